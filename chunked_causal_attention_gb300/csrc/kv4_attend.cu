// Attention of the newest tokens over the 4-bit cache.
//
//   s_rj = scale q_r . k_j,   O_r = sum_j 2^(s2_rj - m_r) v_j / l_r,   s2 = s log2 e
//
// A row of the call is one query of one head; the G = H / Hkv heads that share a
// key/value head and the T new tokens make R = G T rows that read the same slots.
// For few rows the call is bound by the bytes of the cache (0.5625 B a value), so
// every byte is read once, by bulk copies into shared memory, and R rows share it.
//
// Split. The work is the list of 64- or 128-slot tiles of all units (sequence, key/value
// head, group of 8 NT rows). Each block takes an equal stretch of that list, found
// on the device from lens: no block idles whatever the lengths are, and the host
// need not know them. A unit that lies in one block is finished there; the partials
// (O, m, l) of a unit cut between blocks go to the workspace and merge_kernel joins
// them in block order, so results do not depend on timing.
//
// Warps. Each of a block's four warps takes 16 or 32 slots of every tile, with its own
// running maximum and accumulators, and meets the others only at a unit's end. A tile
// is four bulk copies into a stage of shared memory; the last warp to have read a
// stage has it filled again.
//
// Products. With few rows the matrix product's M side is the cache's: S^T = K Q^T
// (16 slots x 8 rows) and O^T = V^T P^T (16 dims x 8 rows), mma m16n8k16 in fp16.
// A value code * scale has at most 6 significant bits, so cvt.rn.f16x2.e2m1x2 and
// one multiplication give it exactly in fp16. Queries are multiplied by a power of
// two that brings the row's largest to [2^14, 2^15): their 8 bits are exact in fp16
// down to 2^-28 of the largest. Which dim stands where in a product is free as long
// as both sides agree, so each lane reads whole words of codes: for K lane c of a
// quad holds a quarter of the row's words, for V^T lane g of the eight row groups
// holds an eighth, and two slots' words are interleaved by two logical operations
// into bytes that convert to (slot a, slot b) pairs.
//
// Measured (128 dims, 4 or 5 rows a head): 1M slots of 8 heads 225 us (5.4 TB/s, 79% of
// the copy rate), 4 x 128K slots 118 us, 1000 slots 9.3 us. 279 instructions for 16 slots
// of keys and values (128 of them conversions and multiplications) keep the issue slots
// 56% and the ALU pipe 49% busy with four warps a scheduler; three blocks an SM are 4%
// slower, five or more spill or wait, 16 slots a step 22% slower.
//
// Softmax weights are rounded to fp16 too, after a factor 2^11 and with a running
// maximum that may lag by up to 2^4: weights stay below 2^15, and those under 2^-35
// of the row's largest are flushed (1M of them would be 2^-15 of the sum). l is
// summed in fp32, one partial sum a lane.
#include <algorithm>
#include <type_traits>

#include "kv4_device.cuh"
#include "tc_common.cuh"

namespace attn {
namespace {

using namespace kv4;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSlots = 16;                 // slots of a fragment; a warp's slice is one or two of them
constexpr float kLag = 4.f;                // how far (log2) a score may pass the running maximum
constexpr float kUp = 11.f;                // weights are held times 2^kUp
constexpr int kMaxGrid = 1024;            // blocks of the split kernel
constexpr int64_t kScores = 1 << 28;       // scores (mass) that a pass keeps, if it has more than one unit a head

// What the launch derives from the shapes.
struct Split {
    int32_t R;            // rows of a key/value head
    int32_t rt0, RT;      // of the units that they make, those of this pass: the first and how many
    int32_t pitch;        // fp32 scores kept of each slot (mass), a row group
    int64_t slot_floats;  // floats of a partial: 8 NT rows of D, then m and l of each
    float* lse2;          // [B H T] log2 of the rows' sums (mass)
    float* scores;        // [unit][cap][pitch]
    uint64_t wait_ns;
    int32_t stall;
};

__host__ __device__ constexpr int blocks_per_sm(int dt, int nt) { return nt > 1 ? 2 : dt <= 128 ? 4 : 3; }

// Fragments of 16 slots in a warp's slice: two where the registers of a second one are there.
__host__ __device__ constexpr int fragments(int dt, int nt) { return nt == 1 && dt <= 128 ? 2 : 1; }
__host__ __device__ constexpr int tile_slots(int dt, int nt) { return kWarps * kSlots * fragments(dt, nt); }

template <int DT, int NT>
struct Layout {
    static constexpr int KS = fragments(DT, NT), SLOTS = kSlots * KS, TILE = tile_slots(DT, NT);
    static constexpr int STAGES = KS == 2 ? 2 : DT == 256 ? 3 : 4;
    static constexpr int CODES = TILE * DT / 2, SCALES = TILE * DT / 16;   // of K; then V's
    static constexpr int STAGE = 2 * (CODES + SCALES);
    static constexpr int RING = STAGES * STAGE;
    static constexpr int ROWS = 8 * NT;
    static constexpr int O_PITCH = DT + 8;
    static constexpr int O_OFF = RING;
    static constexpr int Q_OFF = O_OFF + ROWS * O_PITCH * 4;
    static constexpr bool Q_REGS = NT == 1 && DT <= 128;            // the queries' fragments stay in registers
    static constexpr int Q_BYTES = Q_REGS ? 0 : NT * (DT / 16) * 32 * 8;
    static constexpr int QS_OFF = Q_OFF + Q_BYTES;                  // score factor of each row
    static constexpr int ML_OFF = QS_OFF + ROWS * 4;               // m then l of each warp and row
    static constexpr int BAR_OFF = ML_OFF + 2 * kWarps * ROWS * 4;
    static constexpr int DONE_OFF = BAR_OFF + STAGES * 8;    // of each stage: warps that have read it, times it was filled
    static constexpr int MISC_OFF = DONE_OFF + STAGES * 8;
    static constexpr int BYTES = MISC_OFF + 64;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

// The bits of a where m is set, of b elsewhere.
__device__ __forceinline__ uint32_t pick(uint32_t m, uint32_t a, uint32_t b) { return (a & m) | (b & ~m); }

// Slots in use of sequence b.
__device__ __forceinline__ int32_t slots_of(const Kv4AttendArgs& a, int32_t b) {
    const int64_t most = a.mass_out && a.mass_ld < a.c.cap ? a.mass_ld : a.c.cap;
    return length_of(a.lens, b, (int32_t)most, a.status);
}

template <int TILE>
__device__ __forceinline__ int32_t tiles_of(int32_t n) { return (n + TILE - 1) / TILE; }

// a / b, both not negative, by a 32-bit division where it does (a third of the time).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    return (((uint64_t)a | (uint64_t)b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// First tile of block c when `total` tiles are dealt to `blocks` blocks.
__device__ __forceinline__ int64_t first_tile(int64_t c, int64_t total, int32_t blocks) { return divide(c * total, blocks); }

// The block that holds tile x.
__device__ __forceinline__ int32_t block_of(int64_t x, int64_t total, int32_t blocks) {
    return (int32_t)divide((x + 1) * blocks - 1, total);
}

// Block-wide sums over the sequences of their tiles: of all, and of those before sequence `upto`.
template <int THREADS, int TILE>
__device__ __forceinline__ void sum_tiles(const Kv4AttendArgs& a, int32_t upto, int64_t& total, int64_t& before,
                                          int64_t* scratch) {
    int64_t all = 0, some = 0;
    for (int b = threadIdx.x; b < a.c.B; b += THREADS) {
        const int32_t t = tiles_of<TILE>(slots_of(a, b));
        all += t;
        if (b < upto) some += t;
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, m);
        some += __shfl_xor_sync(0xffffffffu, some, m);
    }
    if ((threadIdx.x & 31) == 0) {
        scratch[2 * (threadIdx.x >> 5)] = all;
        scratch[2 * (threadIdx.x >> 5) + 1] = some;
    }
    __syncthreads();
    total = before = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        total += scratch[2 * w];
        before += scratch[2 * w + 1];
    }
    __syncthreads();
}

// A place in the tile list.
struct Cursor {
    int32_t b, v, t;      // sequence, unit of the sequence, tile of the unit
    int32_t n, nt;        // the sequence's slots in use and tiles
    // The next tile; true if it is another unit's.
    template <int TILE>
    __device__ __forceinline__ bool next(const Kv4AttendArgs& a, int32_t units) {
        if (++t < nt) return false;
        t = 0;
        if (++v < units) return true;
        v = 0;
        nt = 0;
        while (nt == 0 && ++b < a.c.B) {
            n = slots_of(a, b);
            nt = tiles_of<TILE>(n);
        }
        return true;
    }
};

// The words (8 codes each) of a row that a lane holds for the K product: word i of lane c of the quad.
template <int DT>
__device__ __forceinline__ int k_word(int c, int i) {
    return DT == 256 ? (i & 4) * 4 + 4 * c + (i & 3) : (DT / 32) * c + i;
}

template <int DT, int NT, bool EXACT, bool MASS>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(DT, NT)) split_kernel(const Kv4AttendArgs a, const Split sp) {
    using L = Layout<DT, NT>;
    constexpr int KS = L::KS;
    constexpr int KW = DT / 32;            // K words a lane and row
    constexpr int KB = DT / 64;            // K scales a lane and row
    constexpr int VB = DT / 16;            // V bytes a lane and slot = 16-dim steps of O^T
    constexpr int VW = VB / 4;             // V words a lane and slot
    constexpr int VS = DT == 256 ? 2 : 1;  // V scales a lane and slot
    extern __shared__ __align__(128) uint8_t sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    const int cb = EXACT ? DT / 2 : a.c.cb, nb = EXACT ? DT / 16 : a.c.nb, D = EXACT ? DT : a.c.D;
    const int G = a.g.H / a.c.Hkv, units = a.c.Hkv * sp.RT;
    float* sO = reinterpret_cast<float*>(sm + L::O_OFF);
    uint2* sQ = reinterpret_cast<uint2*>(sm + L::Q_OFF);
    float* sQS = reinterpret_cast<float*>(sm + L::QS_OFF);
    float* sM = reinterpret_cast<float*>(sm + L::ML_OFF);
    float* sL = sM + kWarps * L::ROWS;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC_OFF);
    int64_t* scratch = reinterpret_cast<int64_t*>(sm + L::O_OFF);
    const uint32_t ring = smem_u32(sm), bar = ring + L::BAR_OFF;
    uint32_t* done = reinterpret_cast<uint32_t*>(sm + L::DONE_OFF);
    volatile uint32_t* filled = done + L::STAGES;

    if (tid == 0) {
        for (int s = 0; s < L::STAGES; ++s) {
            tc::mbar_init(bar + 8 * s, 1);
            done[s] = 0;
            filled[s] = 0;
        }
        *abort_flag = 0;
        tc::fence_barrier_init();
    }

    grid_wait();
    grid_go();

    // ---- this block's stretch of the tile list
    int64_t total, before;
    sum_tiles<kThreads, L::TILE>(a, 0, total, before, scratch);
    total *= units;
    const int32_t blocks = (int32_t)min((int64_t)a.grid, total);
    if ((int32_t)blockIdx.x >= blocks) return;
    const int64_t t0 = first_tile(blockIdx.x, total, blocks);
    const int32_t n_tiles = (int32_t)(first_tile(blockIdx.x + 1, total, blocks) - t0);
    Cursor cur{0, 0, 0, 0, 0};
    {
        // the sequence that holds tile t0: a scan over as many sequences as there are threads, until it is among them
        int64_t left = t0;
        for (int base = 0;; base += kThreads) {         // t0 < total: there is one
            const int32_t mine = base + tid < a.c.B ? tiles_of<L::TILE>(slots_of(a, base + tid)) : 0;
            int64_t upto = (int64_t)mine * units;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, upto, m);
                if (lane >= m) upto += y;
            }
            if (lane == 31) scratch[warp] = upto;
            __syncthreads();
            int64_t chunk = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) upto += scratch[w];
                chunk += scratch[w];
            }
            if (left < upto && left >= upto - (int64_t)mine * units) {
                scratch[kWarps] = base + tid;
                scratch[kWarps + 1] = left - (upto - (int64_t)mine * units);
            }
            __syncthreads();
            if (left < chunk) break;
            left -= chunk;
            if (base + kThreads >= a.c.B) return;       // lens changed under the kernel: nothing is addressed
        }
        cur.b = (int32_t)scratch[kWarps];
        left = scratch[kWarps + 1];
        cur.n = slots_of(a, cur.b);
        cur.nt = tiles_of<L::TILE>(cur.n);
        cur.v = (int32_t)divide(left, max(cur.nt, 1));
        cur.t = (int32_t)(left - (int64_t)cur.v * cur.nt);
        __syncthreads();                                // scratch is read
    }

    // ---- bulk copies of the tiles, in list order. Every warp follows the cursor; a stage is
    // filled again by the warp that is the last to have read it
    Cursor ahead = cur;
    int64_t ahead_row = 0;                              // cache row of slot 0 of the unit ahead
    auto unit_row = [&]() { ahead_row = (int64_t)ahead.b * a.c.sb + (int64_t)(ahead.v / sp.RT) * a.c.sh; };
    unit_row();
    auto issue = [&](uint32_t s) {                      // one thread
        const int32_t k0 = ahead.t * L::TILE;
        const int64_t row = ahead_row + k0;
        const uint32_t dst = ring + s * L::STAGE, f = bar + 8 * s;
        // no further than the 16 slots that hold the last one (the capacity is a multiple of 16)
        const uint32_t slots = min(L::TILE, (ahead.n - k0 + kSlots - 1) & ~(kSlots - 1));
        const uint32_t nc = slots * cb, ns = slots * nb;
        filled[s] = filled[s] + 1;
        tc::mbar_expect_tx(f, 2 * (nc + ns));
        bulk_load(dst, a.c.kc + row * cb, nc, f);
        bulk_load(dst + 2 * L::CODES, a.c.ks + row * nb, ns, f);
        bulk_load(dst + L::CODES, a.c.vc + row * cb, nc, f);
        bulk_load(dst + 2 * L::CODES + L::SCALES, a.c.vs + row * nb, ns, f);
    };
    bool ok = true;
    int32_t to_fetch = n_tiles;
#pragma unroll
    for (int s = 0; s < L::STAGES; ++s)
        if (to_fetch > 0) {
            if (tid == 0 && !sp.stall) issue(s);
            if (--to_fetch > 0 && ahead.next<L::TILE>(a, units)) unit_row();
        }
    uint32_t stage = 0, parity = 0;

    // slot of a 16-row fragment row: neighbours in a different half of a bank line for K's and V's reads
    const int slot_lo = g ^ ((g >> 1) & 1);
    // the fragment's columns 2c, 2c+1 (and 8 further): the same permutation
    const int v_even = (2 * c) ^ (c & 1), v_odd = (2 * c + 1) ^ (c & 1);

    uint32_t qf[L::Q_REGS ? DT / 16 : 1][2];
    float qs[NT][2], l[NT][2];
    float up[NT][2];                                    // kUp - m, m the running maximum
    int32_t lim[NT][2];                                 // slots [0, lim) seen
    int32_t lim_min = 0;                                // by every row
    int32_t hk = 0, rt = 0;
    float o[NT][VB][4];
    bool fresh = true;

    for (int32_t it = 0; it < n_tiles; ++it) {
        if (fresh) {
            // ---- a unit begins: its queries
            fresh = false;
            hk = cur.v / sp.RT;
            rt = sp.rt0 + cur.v - hk * sp.RT;
            __syncthreads();                            // the last unit's sO, sQ, sQS are read
            const int rows = min(L::ROWS, sp.R - rt * L::ROWS);
#pragma unroll 1
            for (int n = 0; n < NT; ++n) {
                if (!L::Q_REGS && (n & (kWarps - 1)) != warp) continue;
                const int r = rt * L::ROWS + 8 * n + g;
                const bool on = 8 * n + g < rows;
                const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + (int64_t)cur.b * a.g.sb +
                                         (int64_t)(hk * G + r % G) * a.g.sh + (int64_t)(r / G) * a.g.st;
                uint32_t w[KW][4];
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < KW; ++i) {
                    const int kw = k_word<DT>(c, i);
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (on && 8 * kw < D) x = *reinterpret_cast<const uint4*>(q + 8 * kw);
                    w[i][0] = x.x; w[i][1] = x.y; w[i][2] = x.z; w[i][3] = x.w;
#pragma unroll
                    for (int j = 0; j < 4; ++j) top = max(top, max(w[i][j] & 0x7FFFu, (w[i][j] >> 16) & 0x7FFFu));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^(14 - e), e the largest's exponent; 1 for a row of zeros or with a value that is not finite
                int lift = 14 - ((int)(top >> 7) - 127);
                lift = min(lift, 120);
                if (top == 0 || top >= 0x7F80u) lift = 0;
                const float f = __int_as_float((127 + lift) << 23);
                if (c == 0 && (!L::Q_REGS || warp == 0))
                    sQS[8 * n + g] = a.g.scale * kLog2e * __int_as_float((127 - lift) << 23) * a.c.k_scale;
#pragma unroll
                for (int i = 0; i < KW; ++i)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t p[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t x = w[i][2 * half + j];
                            p[j] = as_u32(__floats2half2_rn(__uint_as_float(x << 16) * f,
                                                            __uint_as_float(x & 0xFFFF0000u) * f));
                        }
                        if constexpr (L::Q_REGS) {
                            qf[2 * i + half][0] = p[0];
                            qf[2 * i + half][1] = p[1];
                        } else {
                            sQ[(n * (DT / 16) + 2 * i + half) * 32 + lane] = make_uint2(p[0], p[1]);
                        }
                    }
            }
            __syncthreads();
            lim_min = cur.n - a.g.T + 1 + (rt * L::ROWS) / G;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = 8 * n + 2 * c + j;
                    qs[n][j] = sQS[r];
                    lim[n][j] = r < rows ? cur.n - a.g.T + 1 + (rt * L::ROWS + r) / G : 0;
                    up[n][j] = INFINITY;
                    l[n][j] = 0.f;
                }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < VB; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
        }

        // every warp waits for every tile, also one it has no slots of: a parity tells neighbouring phases apart only
        if (ok) ok = tc::mbar_wait_warp(bar + 8 * stage, parity, abort_flag, a.status, sp.wait_ns);
        const int32_t k0 = cur.t * L::TILE + warp * L::SLOTS;
        if (k0 < cur.n && ok) {
            const uint8_t* slice = sm + stage * L::STAGE + warp * L::SLOTS * cb;                 // codes
            const uint8_t* slice_s = sm + stage * L::STAGE + 2 * L::CODES + warp * L::SLOTS * nb;  // scales
            // the slots that some row does not see are few: a copy of the code of their own
            auto work = [&](auto masked_) {
                constexpr bool masked = decltype(masked_)::value;
                // ---- S^T = K Q^T
                float s[KS][NT][4];
#pragma unroll
                for (int x = 0; x < KS; ++x) {
                    const uint8_t* kc = slice + x * kSlots * cb;
                    const uint8_t* ks = slice_s + x * kSlots * nb;
                    uint32_t kw[2][KW];
                    uint32_t ksc[2][KB];                // scale of each block, in both halves
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = slot_lo + 8 * h;
                        if constexpr (EXACT) {
                            if constexpr (DT == 64) {
                                const uint2 w = *reinterpret_cast<const uint2*>(kc + r * 32 + 8 * c);
                                kw[h][0] = w.x; kw[h][1] = w.y;
                                ksc[h][0] = __byte_perm(scales_f16x2(ks[r * 4 + c]), 0, 0x1010);
                            } else {
#pragma unroll
                                for (int p = 0; p < DT / 128; ++p) {
                                    const uint4 w = *reinterpret_cast<const uint4*>(kc + r * (DT / 2) + 64 * p + 16 * c);
                                    kw[h][4 * p] = w.x; kw[h][4 * p + 1] = w.y; kw[h][4 * p + 2] = w.z; kw[h][4 * p + 3] = w.w;
                                    const uint32_t y = scales_f16x2(
                                        *reinterpret_cast<const uint16_t*>(ks + r * (DT / 16) + 8 * p + 2 * c));
                                    ksc[h][2 * p] = __byte_perm(y, 0, 0x1010);
                                    ksc[h][2 * p + 1] = __byte_perm(y, 0, 0x3232);
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < KW; ++i) {
                                const int wd = k_word<DT>(c, i);
                                kw[h][i] = 8 * wd < D ? *reinterpret_cast<const uint32_t*>(kc + r * cb + 4 * wd) : 0u;
                                if (!(i & 1))
                                    ksc[h][i / 2] = __byte_perm(scales_f16x2(8 * wd < D ? ks[r * nb + wd / 2] : 0), 0, 0x1010);
                            }
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[x][n][j] = 0.f;
#pragma unroll
                    for (int i = 0; i < KW; ++i) {
                        const __half2 s0 = as_half2(ksc[0][i / 2]), s1 = as_half2(ksc[1][i / 2]);
                        const uint32_t x0 = kw[0][i], x1 = kw[1][i];
                        const uint32_t a0[4] = {as_u32(__hmul2(as_half2(codes_f16x2<0>(x0)), s0)),
                                                as_u32(__hmul2(as_half2(codes_f16x2<0>(x1)), s1)),
                                                as_u32(__hmul2(as_half2(codes_f16x2<1>(x0)), s0)),
                                                as_u32(__hmul2(as_half2(codes_f16x2<1>(x1)), s1))};
                        const uint32_t a1[4] = {as_u32(__hmul2(as_half2(codes_f16x2<2>(x0)), s0)),
                                                as_u32(__hmul2(as_half2(codes_f16x2<2>(x1)), s1)),
                                                as_u32(__hmul2(as_half2(codes_f16x2<3>(x0)), s0)),
                                                as_u32(__hmul2(as_half2(codes_f16x2<3>(x1)), s1))};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if constexpr (L::Q_REGS) {
                                mma16816(s[x][n], a0, qf[2 * i][0], qf[2 * i][1]);
                                mma16816(s[x][n], a1, qf[2 * i + 1][0], qf[2 * i + 1][1]);
                            } else {
                                const uint2 b0 = sQ[(n * (DT / 16) + 2 * i) * 32 + lane];
                                const uint2 b1 = sQ[(n * (DT / 16) + 2 * i + 1) * 32 + lane];
                                mma16816(s[x][n], a0, b0.x, b0.y);
                                mma16816(s[x][n], a1, b1.x, b1.y);
                            }
                        }
                    }
                }

                // ---- weights: 2^(s qs + kUp - m)
                const int ka = k0 + slot_lo;            // this lane's slots: ka + 16 x, and 8 further
                if constexpr (MASS) {
                    float* dst = sp.scores + ((int64_t)(cur.b * units + cur.v) * a.c.cap + ka) * sp.pitch + 2 * c;
#pragma unroll
                    for (int x = 0; x < KS; ++x)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            if (8 * n + 2 * c < sp.pitch)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const int k = ka + kSlots * x + 8 * h;
                                    if (k < cur.n)
                                        *reinterpret_cast<float2*>(dst + 8 * n + (int64_t)(kSlots * x + 8 * h) * sp.pitch) =
                                            make_float2(k < lim[n][0] ? s[x][n][2 * h] * qs[n][0] : -INFINITY,
                                                        k < lim[n][1] ? s[x][n][2 * h + 1] * qs[n][1] : -INFINITY);
                                }
                }
                float e[KS][NT][4];
                float most = -INFINITY;
#pragma unroll
                for (int x = 0; x < KS; ++x)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            // product and sum rounded apart, so that the maximum's own exponent is exact at any size
                            const float2 y = tc::fadd2(tc::fmul2(make_float2(s[x][n][2 * h], s[x][n][2 * h + 1]),
                                                                 make_float2(qs[n][0], qs[n][1])),
                                                       make_float2(up[n][0], up[n][1]));
                            e[x][n][2 * h] = y.x;
                            e[x][n][2 * h + 1] = y.y;
                        }
                if (masked) {
#pragma unroll
                    for (int x = 0; x < KS; ++x)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (ka + kSlots * x + (j & 2) * 4 >= lim[n][j & 1]) e[x][n][j] = -INFINITY;
                }
#pragma unroll
                for (int x = 0; x < KS; ++x)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; j += 2) most = tc::fmax3(most, e[x][n][j], e[x][n][j + 1]);
                if (__any_sync(0xffffffffu, most > kUp + kLag)) {
                    // the running maximum moves to this slice's, where that is larger
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float t = -INFINITY;
#pragma unroll
                            for (int x = 0; x < KS; ++x)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    if (!masked || ka + kSlots * x + 8 * h < lim[n][j]) t = fmaxf(t, __fmul_rn(s[x][n][2 * h + j], qs[n][j]));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                            const float was = up[n][j], now = fminf(was, kUp - t);
                            const float f = now == was ? 1.f : ex2(now - was);
                            up[n][j] = now;
                            l[n][j] *= f;
#pragma unroll
                            for (int i = 0; i < VB; ++i) {
                                o[n][i][j] *= f;
                                o[n][i][j + 2] *= f;
                            }
#pragma unroll
                            for (int x = 0; x < KS; ++x)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    float& y = e[x][n][2 * h + j];
                                    // a row that has seen no slot yet (now = inf) has weight 0, or NaN
                                    y = masked && ka + kSlots * x + 8 * h >= lim[n][j]
                                            ? -INFINITY
                                            : __fadd_rn(__fmul_rn(s[x][n][2 * h + j], qs[n][j]), now);
                                }
                        }
                }
                uint32_t p[KS][NT][2];
#pragma unroll
                for (int x = 0; x < KS; ++x)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float p0 = ex2(e[x][n][0]), p1 = ex2(e[x][n][1]), p2 = ex2(e[x][n][2]), p3 = ex2(e[x][n][3]);
                        const float2 y = tc::fadd2(make_float2(l[n][0], l[n][1]),
                                                   tc::fadd2(make_float2(p0, p1), make_float2(p2, p3)));
                        l[n][0] = y.x;
                        l[n][1] = y.y;
                        p[x][n][0] = transpose8(as_u32(__floats2half2_rn(p0, p1)));
                        p[x][n][1] = transpose8(as_u32(__floats2half2_rn(p2, p3)));
                    }

                // ---- O^T += V^T P^T
#pragma unroll
                for (int x = 0; x < KS; ++x) {
                    const uint8_t* vc = slice + L::CODES + x * kSlots * cb;
                    const uint8_t* vs = slice_s + L::SCALES + x * kSlots * nb;
                    uint32_t vw[4][VW];
                    uint32_t vraw[4][VS];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = (i & 1 ? v_odd : v_even) + (i & 2) * 4;
                        if constexpr (EXACT) {
                            const uint8_t* p8 = vc + r * (DT / 2) + VB * g;
                            if constexpr (DT == 64) vw[i][0] = *reinterpret_cast<const uint32_t*>(p8);
                            if constexpr (DT == 128) {
                                const uint2 w = *reinterpret_cast<const uint2*>(p8);
                                vw[i][0] = w.x; vw[i][1] = w.y;
                            }
                            if constexpr (DT == 256) {
                                const uint4 w = *reinterpret_cast<const uint4*>(p8);
                                vw[i][0] = w.x; vw[i][1] = w.y; vw[i][2] = w.z; vw[i][3] = w.w;
                                const uint32_t y = *reinterpret_cast<const uint16_t*>(vs + r * 16 + 2 * g);
                                vraw[i][0] = y & 0xFF;
                                vraw[i][1] = y >> 8;
                            } else {
                                vraw[i][0] = vs[r * (DT / 16) + (DT == 64 ? g >> 1 : g)];
                            }
                        } else {
#pragma unroll
                            for (int w = 0; w < VW; ++w) {
                                const int wd = VW * g + w;
                                vw[i][w] = 8 * wd < D ? *reinterpret_cast<const uint32_t*>(vc + r * cb + 4 * wd) : 0u;
                                if (w % 2 == 0) vraw[i][w / 2] = 8 * wd < D ? vs[r * nb + wd / 2] : 0u;
                            }
                        }
                    }
                    bool nan = false;
                    if (masked) {
                        // slots behind the last one hold anything: scale 0. NaN scales of slots that some
                        // rows do not see are kept out of the product and given to the rows that do
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int y = 0; y < VS; ++y) {
                                if (k0 + kSlots * x + (i & 1 ? v_odd : v_even) + (i & 2) * 4 >= cur.n) vraw[i][y] = 0;
                                if ((vraw[i][y] & 0x7F) == 0x7F) {
                                    nan = true;
                                    vraw[i][y] = 0;
                                }
                            }
                    }
                    uint32_t vsc[2][VS];                // scales of slot pairs
#pragma unroll
                    for (int y = 0; y < VS; ++y) {
                        vsc[0][y] = scales_f16x2(vraw[0][y] | vraw[1][y] << 8);
                        vsc[1][y] = scales_f16x2(vraw[2][y] | vraw[3][y] << 8);
                    }
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        constexpr uint32_t M = 0x0F0F0F0Fu;
                        const uint32_t lo0 = pick(M, vw[0][w], vw[1][w] << 4), hi0 = pick(M, vw[0][w] >> 4, vw[1][w]);
                        const uint32_t lo1 = pick(M, vw[2][w], vw[3][w] << 4), hi1 = pick(M, vw[2][w] >> 4, vw[3][w]);
                        const __half2 s0 = as_half2(vsc[0][w / 2]), s1 = as_half2(vsc[1][w / 2]);
                        auto step = [&](int i, uint32_t l0, uint32_t h0, uint32_t l1, uint32_t h1) {
                            const uint32_t av[4] = {as_u32(__hmul2(as_half2(l0), s0)), as_u32(__hmul2(as_half2(h0), s0)),
                                                    as_u32(__hmul2(as_half2(l1), s1)), as_u32(__hmul2(as_half2(h1), s1))};
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma16816(o[n][4 * w + i], av, p[x][n][0], p[x][n][1]);
                        };
                        step(0, codes_f16x2<0>(lo0), codes_f16x2<0>(hi0), codes_f16x2<0>(lo1), codes_f16x2<0>(hi1));
                        step(1, codes_f16x2<1>(lo0), codes_f16x2<1>(hi0), codes_f16x2<1>(lo1), codes_f16x2<1>(hi1));
                        step(2, codes_f16x2<2>(lo0), codes_f16x2<2>(hi0), codes_f16x2<2>(lo1), codes_f16x2<2>(hi1));
                        step(3, codes_f16x2<3>(lo0), codes_f16x2<3>(hi0), codes_f16x2<3>(lo1), codes_f16x2<3>(hi1));
                    }
                    if (masked && __any_sync(0xffffffffu, nan)) {
#pragma unroll 1
                        for (int k = 0; k < kSlots; ++k) {
                            const int at = k0 + kSlots * x + k;
                            if (at >= cur.n) break;
#pragma unroll
                            for (int w = 0; w < VW; ++w) {
                                const int wd = VW * g + w;
                                if (8 * wd >= D || (vs[k * nb + wd / 2] & 0x7F) != 0x7F) continue;
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int j = 0; j < 4; ++j)
#pragma unroll
                                        for (int i = 0; i < 4; ++i)
                                            if (at < lim[n][j & 1]) o[n][4 * w + i][j] = __int_as_float(0x7FC00000);
                            }
                        }
                    }
                }
            };
            if (k0 + L::SLOTS > lim_min) work(std::true_type{});
            else work(std::false_type{});
        }
        __syncwarp();                                   // the slice is read
        if (to_fetch > 0) {
            if (lane == 0) {
                __threadfence_block();
                // counts to kWarps and back to 0
                if (atomicInc(done + stage, kWarps - 1) == kWarps - 1 && ok && !sp.stall) issue(stage);
            }
            if (--to_fetch > 0 && ahead.next<L::TILE>(a, units)) unit_row();
        }
        if (++stage == L::STAGES) {
            stage = 0;
            parity ^= 1;
        }

        if (cur.t == cur.nt - 1 || it == n_tiles - 1) {
            // ---- the unit, or this block's share of it, ends: join the warps
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = l[n][j];
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    x += __shfl_xor_sync(0xffffffffu, x, 16);
                    if (g == 0) {
                        sM[warp * L::ROWS + 8 * n + 2 * c + j] = kUp - up[n][j];
                        sL[warp * L::ROWS + 8 * n + 2 * c + j] = x;
                    }
                }
            __syncthreads();
            float f[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = 8 * n + 2 * c + j;
                    float top = sM[r];
                    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sM[w * L::ROWS + r]);
                    f[n][j] = up[n][j] == INFINITY ? 0.f : ex2(kUp - up[n][j] - top);
                }
            for (int w = 0; w < kWarps; ++w) {
                if (warp == w) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float2* dst = reinterpret_cast<float2*>(sO + (8 * n + 2 * c + j) * L::O_PITCH + 2 * VB * g);
#pragma unroll
                            for (int i = 0; i < VB; ++i) {
                                float2 x = make_float2(o[n][i][j] * f[n][j], o[n][i][j + 2] * f[n][j]);
                                if (w) x = make_float2(x.x + dst[i].x, x.y + dst[i].y);
                                dst[i] = x;
                            }
                        }
                }
                __syncthreads();
            }
            const int rows = min(L::ROWS, sp.R - rt * L::ROWS);
            const bool begins = it >= cur.t, ends = cur.t == cur.nt - 1;
            float* part = a.parts + (2 * (int64_t)blockIdx.x + (begins ? 1 : 0)) * sp.slot_floats;
            for (int r = warp; r < rows; r += kWarps) {
                float top = sM[r], sum = 0.f;
                for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sM[w * L::ROWS + r]);
                for (int w = 0; w < kWarps; ++w) {
                    const float mw = sM[w * L::ROWS + r];
                    sum += sL[w * L::ROWS + r] * (mw == -INFINITY ? 0.f : ex2(mw - top));
                }
                if (begins && ends) {
                    const int rr = rt * L::ROWS + r, h = hk * G + rr % G, i = rr / G;
                    const bool none = cur.n - a.g.T + 1 + i <= 0;
                    const float inv = none ? 0.f : a.c.v_scale / sum;
                    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.o) + (int64_t)cur.b * a.g.sb +
                                         (int64_t)h * a.g.sh + (int64_t)i * a.g.st;
                    for (int d = 2 * lane; d < D; d += 64)
                        *reinterpret_cast<uint32_t*>(dst + d) = pack_bf16(sO[r * L::O_PITCH + d] * inv, sO[r * L::O_PITCH + d + 1] * inv);
                    if (lane == 0) {
                        const float l2 = none ? -INFINITY : top - kUp + lg2(sum);
                        const int64_t at = ((int64_t)cur.b * a.g.H + h) * a.g.T + i;
                        a.lse[at] = l2 * kLn2;
                        if (MASS) sp.lse2[at] = l2;
                    }
                } else {
                    for (int d = 2 * lane; d < D; d += 64)
                        *reinterpret_cast<float2*>(part + (int64_t)r * D + d) =
                            *reinterpret_cast<const float2*>(sO + r * L::O_PITCH + d);
                    if (lane == 0) {
                        part[(int64_t)L::ROWS * D + r] = top;
                        part[(int64_t)L::ROWS * D + L::ROWS + r] = sum;
                    }
                }
            }
            fresh = true;
        }
        if (it + 1 < n_tiles) cur.next<L::TILE>(a, units);
    }
    // a wait gave up: copies in flight end (bounded) before the block does; no stage is filled after the last unit's barriers
    if (!ok && tid == 0)
        for (int s = 0; s < L::STAGES; ++s) {
            const uint64_t begin = tc::globaltimer();
            while (filled[s] && !tc::mbar_try_wait(bar + 8 * s, (filled[s] - 1) & 1) &&
                   tc::globaltimer() - begin < sp.wait_ns) {
            }
        }
}

// Rows of units that no block finished: the partials of the blocks that share the
// unit, in block order; and the rows of empty sequences. WPR warps take a row, each
// every WPR-th partial, and add up their sums in order: eight where few rows have many
// partials (1 of 8 units of 128K slots lies in 76 blocks), so that their loads are in
// flight together, one where there are many rows. Lanes hold the weights of 32
// partials and four dims each.
constexpr int kMergeWarps = 8;
constexpr int kMergeThreads = 32 * kMergeWarps;
template <int TILE, int WPR>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const Kv4AttendArgs a, const Split sp, int32_t unit_rows) {
    constexpr int ROWS = kMergeWarps / WPR;             // of a block
    __shared__ int64_t scratch[2 * kMergeWarps];
    __shared__ int32_t range[3];
    __shared__ float red[2][kMergeWarps];
    __shared__ __align__(16) float sums[WPR == 1 ? 1 : kMergeWarps][WPR == 1 ? 4 : 256];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, part = warp % WPR;
    const int G = a.g.H / a.c.Hkv, units = a.c.Hkv * sp.RT, groups = unit_rows / ROWS;
    const int u = blockIdx.x / groups, r = (blockIdx.x - u * groups) * ROWS + warp / WPR;
    const int b = u / units, v = u - b * units, hk = v / sp.RT, rt = sp.rt0 + v - hk * sp.RT;
    const int rr = rt * unit_rows + r;
    const int i = rr / G, h = hk * G + rr - i * G, D = a.c.D;
    // every block waits for the kernel before, so that this one does not end ahead of it
    if (rt * unit_rows + (blockIdx.x - u * groups) * ROWS >= sp.R) {            // no row of the block is one
        grid_wait();
        grid_go();
        return;
    }
    const int32_t n = slots_of(a, b);
    int64_t total, before;
    sum_tiles<kMergeThreads, TILE>(a, b, total, before, scratch);
    if (tid == 0) {
        total *= units;
        const int32_t blocks = (int32_t)min((int64_t)a.grid, total), nt = tiles_of<TILE>(n);
        const int64_t first = before * units + (int64_t)v * nt;
        range[0] = nt ? block_of(first, total, blocks) : 0;
        range[1] = nt ? block_of(first + nt - 1, total, blocks) : 0;
    }
    grid_wait();                                        // the split kernel's partials
    grid_go();
    __syncthreads();
    const int c0 = range[0], c1 = range[1];
    const bool row = rr < sp.R, none = n - a.g.T + 1 + i <= 0;
    const int64_t at = ((int64_t)b * a.g.H + h) * a.g.T + i;
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.o) + (int64_t)b * a.g.sb + (int64_t)h * a.g.sh +
                         (int64_t)i * a.g.st;
    if (row && none && part == 0) {
        for (int d = lane; d < D; d += 32) dst[d] = __float2bfloat16(0.f);
        if (lane == 0) {
            a.lse[at] = -INFINITY;
            if (sp.lse2) sp.lse2[at] = -INFINITY;
        }
    }
    if (c0 == c1) return;                               // finished by its block; the same for the whole block
    // block c0 holds the unit's begin: there the partial is the block's second
    auto slot = [&](int c) { return a.parts + (2 * (int64_t)c + (c == c0 ? 1 : 0)) * sp.slot_floats; };
    const int64_t off_m = (int64_t)unit_rows * D + r, off_l = off_m + unit_rows;
    const bool live = row && !none;
    float top = -INFINITY;
    if (live)
        for (int c = c0 + part + WPR * lane; c <= c1; c += WPR * 32) top = fmaxf(top, slot(c)[off_m]);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    if (WPR > 1) {
        if (lane == 0) red[0][warp] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WPR; ++w) top = fmaxf(top, red[0][warp - part + w]);
    }
    float sum = 0.f;
    float4 y[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (live)
        for (int base = c0 + part; base <= c1; base += WPR * 32) {
            const int mine = base + WPR * lane;
            float w = 0.f;
            if (mine <= c1) {
                const float mc = slot(mine)[off_m];
                w = mc == -INFINITY ? 0.f : ex2(mc - top);
                sum += w * slot(mine)[off_l];
            }
            const int count = min(32, (c1 - base) / WPR + 1);
#pragma unroll 8
            for (int k = 0; k < count; ++k) {
                const float f = __shfl_sync(0xffffffffu, w, k);
                const float* p = slot(base + WPR * k) + (int64_t)r * D + 4 * lane;
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (4 * lane + 128 * x < D) {
                        const float4 z = *reinterpret_cast<const float4*>(p + 128 * x);
                        y[x] = make_float4(fmaf(f, z.x, y[x].x), fmaf(f, z.y, y[x].y), fmaf(f, z.z, y[x].z), fmaf(f, z.w, y[x].w));
                    }
            }
        }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (WPR > 1) {
        if (lane == 0) red[1][warp] = sum;
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (4 * lane + 128 * x < D) *reinterpret_cast<float4*>(&sums[warp][4 * lane + 128 * x]) = y[x];
        __syncthreads();
        if (part) return;
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) sum += red[1][warp + w];
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (4 * lane + 128 * x < D) {
                y[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < WPR; ++w) {
                    const float4 z = *reinterpret_cast<const float4*>(&sums[warp + w][4 * lane + 128 * x]);
                    y[x] = make_float4(y[x].x + z.x, y[x].y + z.y, y[x].z + z.z, y[x].w + z.w);
                }
            }
    }
    if (!live) return;
    const float inv = a.c.v_scale / sum;
#pragma unroll
    for (int x = 0; x < 2; ++x)
        if (4 * lane + 128 * x < D)
            *reinterpret_cast<uint2*>(dst + 4 * lane + 128 * x) =
                make_uint2(pack_bf16(y[x].x * inv, y[x].y * inv), pack_bf16(y[x].z * inv, y[x].w * inv));
    if (lane == 0) {
        const float l2 = top - kUp + lg2(sum);
        a.lse[at] = l2 * kLn2;
        if (sp.lse2) sp.lse2[at] = l2;
    }
}

// mass_out = mass_in + sum over the rows of 2^(s2 - lse2), from the scores that the
// split kernel kept; a thread takes kMassSlots slots, kMassThreads apart, V scores of
// a slot at a time. What it reads before its wait, the weights so far, the pass before may
// have written: older than the split and merge kernels between.
constexpr int kMassThreads = 256, kMassSlots = 4;
template <int V>
__global__ void __launch_bounds__(kMassThreads) mass_kernel(const Kv4AttendArgs a, const Split sp, int32_t unit_rows) {
    __shared__ float s_lse[32];
    const int chunks = (a.c.cap + kMassThreads * kMassSlots - 1) / (kMassThreads * kMassSlots);
    const int bh = blockIdx.x / chunks, b = bh / a.c.Hkv, hk = bh - b * a.c.Hkv, G = a.g.H / a.c.Hkv;
    const int32_t n = slots_of(a, b);
    const int j0 = (blockIdx.x - bh * chunks) * kMassThreads * kMassSlots + threadIdx.x;
    if (j0 - (int)threadIdx.x >= n) {
        grid_wait();
        grid_go();
        return;
    }
    float sum[kMassSlots], base[kMassSlots];
    const int64_t at = (int64_t)bh * a.mass_ld + j0;
#pragma unroll
    for (int x = 0; x < kMassSlots; ++x) {
        sum[x] = 0.f;
        base[x] = a.mass_in && j0 + x * kMassThreads < n ? a.mass_in[at + x * kMassThreads] : 0.f;
    }
    grid_wait();                                        // scores and sums
    grid_go();
    for (int rt = 0; rt < sp.RT; ++rt) {
        __syncthreads();
        if (threadIdx.x < sp.pitch) {
            // rows that see nothing, and columns past the rows, weigh nothing
            const int rr = (sp.rt0 + rt) * unit_rows + threadIdx.x;
            float l2 = rr < sp.R ? sp.lse2[((int64_t)b * a.g.H + hk * G + rr % G) * a.g.T + rr / G] : INFINITY;
            s_lse[threadIdx.x] = l2 == -INFINITY ? INFINITY : l2;
        }
        __syncthreads();
        const float* s = sp.scores + ((int64_t)((int64_t)bh * sp.RT + rt) * a.c.cap + j0) * sp.pitch;
        for (int r = 0; r < sp.pitch; r += V) {
            float y[kMassSlots][V];
#pragma unroll
            for (int x = 0; x < kMassSlots; ++x)
                if (j0 + x * kMassThreads < n) {
                    const float* p = s + (int64_t)x * kMassThreads * sp.pitch + r;
                    if constexpr (V == 4) *reinterpret_cast<float4*>(y[x]) = *reinterpret_cast<const float4*>(p);
                    else *reinterpret_cast<float2*>(y[x]) = *reinterpret_cast<const float2*>(p);
                }
#pragma unroll
            for (int x = 0; x < kMassSlots; ++x)
                if (j0 + x * kMassThreads < n)
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[x] += ex2(y[x][i] - s_lse[r + i]);
        }
    }
#pragma unroll
    for (int x = 0; x < kMassSlots; ++x)
        if (j0 + x * kMassThreads < n) a.mass_out[at + x * kMassThreads] = base[x] + sum[x];
}

// Groups of 8 rows that share a pass over the slots. Four of them save conversions, but
// leave two blocks of 255 registers on an SM: at D = 128 and 32 rows 224 against 248 us
// for 4 sequences of 64K slots and 8 heads, 44 against 29 us for 2K slots, and two groups
// were no faster than one at any size. So four only for at least 32 rows and long caches;
// above 128 dims two (252 registers already with one).
int row_groups(int D, int64_t R, int64_t slots) {
    if (D > 128) return R <= 8 ? 1 : 2;
    return R >= 32 && slots >= (int64_t)1 << 20 ? 4 : 1;
}

int dims_of(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

struct Plan {
    int nt, tile, grid;
    int units;                        // of 8 nt rows, of a key/value head; sp.RT of them a pass
    Split sp;
    int64_t parts, lse2, scores;      // floats
};

Plan plan_of(const Kv4Geom& c, const Geom& g, bool mass) {
    Plan p;
    const int64_t R = (int64_t)(g.H / c.Hkv) * g.T;
    p.nt = row_groups(c.D, R, (int64_t)c.B * c.Hkv * c.cap);
    p.sp.R = (int32_t)R;
    p.units = (int32_t)((R + 8 * p.nt - 1) / (8 * p.nt));
    p.sp.rt0 = 0;
    p.sp.RT = p.units;
    p.sp.pitch = R <= 2 ? 2 : R <= 4 ? 4 : 8 * p.nt;
    if (mass) {
        // each unit goes over the cache by itself, so passes cost their launches only, against a pass's work on
        // 1 GiB of scores (8 heads of 128K slots: 256 rows of each)
        const int64_t most = std::max<int64_t>(1, kScores / ((int64_t)c.B * c.Hkv * c.cap * p.sp.pitch));
        const int64_t passes = (p.units + most - 1) / most;
        p.sp.RT = (int32_t)((p.units + passes - 1) / passes);
    }
    p.sp.slot_floats = (int64_t)8 * p.nt * (c.D + 2);
    const int64_t units = (int64_t)c.B * c.Hkv * p.sp.RT;
    p.tile = tile_slots(dims_of(c.D), p.nt);
    const int64_t tiles = units * ((c.cap + p.tile - 1) / p.tile);
    p.grid = (int)std::min<int64_t>(std::min(device_sm_count() * blocks_per_sm(dims_of(c.D), p.nt), kMaxGrid), tiles);
    p.parts = 2 * (int64_t)p.grid * p.sp.slot_floats;
    p.lse2 = mass ? ((int64_t)g.B * g.H * g.T + 63) / 64 * 64 : 0;
    p.scores = mass ? units * c.cap * p.sp.pitch : 0;
    return p;
}

template <int DT, int NT, bool EXACT, bool MASS>
cudaError_t launch_split(const Kv4AttendArgs& a, const Plan& p, cudaStream_t s) {
    constexpr int bytes = Layout<DT, NT>::BYTES;
    if (bytes > 48 * 1024) {                     // what a block may have without asking
        const cudaError_t e =
            cudaFuncSetAttribute(split_kernel<DT, NT, EXACT, MASS>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    return launch_early(split_kernel<DT, NT, EXACT, MASS>, dim3(p.grid), kThreads, bytes, 1, s, a, p.sp);
}

template <int DT, int NT>
cudaError_t launch_dims(const Kv4AttendArgs& a, const Plan& p, cudaStream_t s) {
    if (a.c.D == DT) return a.mass_out ? launch_split<DT, NT, true, true>(a, p, s) : launch_split<DT, NT, true, false>(a, p, s);
    return a.mass_out ? launch_split<DT, NT, false, true>(a, p, s) : launch_split<DT, NT, false, false>(a, p, s);
}

}  // namespace

size_t kv4_attend_bytes(const Kv4Geom& c, const Geom& g, bool mass) {
    const Plan p = plan_of(c, g, mass);
    return (size_t)(p.parts + p.lse2 + p.scores) * 4;
}

cudaError_t launch_kv4_attend(const Kv4AttendArgs& args, cudaStream_t s) {
    Kv4AttendArgs a = args;
    Plan p = plan_of(a.c, a.g, a.mass_out != nullptr);
    a.grid = p.grid;
    p.sp.lse2 = a.mass_out ? a.parts + p.parts : nullptr;
    p.sp.scores = a.mass_out ? a.parts + p.parts + p.lse2 : nullptr;
    wait_settings(&p.sp.wait_ns, &p.sp.stall);
    const int unit_rows = 8 * p.nt;
    for (int32_t RT = p.sp.RT; p.sp.rt0 < p.units; p.sp.rt0 += RT) {
        p.sp.RT = std::min(RT, p.units - p.sp.rt0);
        if (p.sp.rt0) a.mass_in = a.mass_out;
        cudaError_t e;
        if (a.c.D <= 64) e = p.nt == 1 ? launch_dims<64, 1>(a, p, s) : launch_dims<64, 4>(a, p, s);
        else if (a.c.D <= 128) e = p.nt == 1 ? launch_dims<128, 1>(a, p, s) : launch_dims<128, 4>(a, p, s);
        else e = p.nt == 1 ? launch_dims<256, 1>(a, p, s) : launch_dims<256, 2>(a, p, s);
        if (e != cudaSuccess) return e;
        const int64_t units = (int64_t)a.c.B * a.c.Hkv * p.sp.RT;
        // eight warps a row while that leaves the SMs fewer than two blocks each
        const bool few = units * std::min(unit_rows, p.sp.R) <= 2 * device_sm_count();
        e = launch_early(few ? (p.tile == 128 ? merge_kernel<128, 8> : merge_kernel<64, 8>)
                             : (p.tile == 128 ? merge_kernel<128, 1> : merge_kernel<64, 1>),
                         dim3((unsigned)(units * unit_rows / (few ? 1 : kMergeWarps))), kMergeThreads, 0, 1, s, a, p.sp, unit_rows);
        if (e != cudaSuccess) return e;
        if (!a.mass_out) continue;
        constexpr int per = kMassThreads * kMassSlots;
        e = launch_early(p.sp.pitch % 4 ? mass_kernel<2> : mass_kernel<4>,
                         dim3((unsigned)((int64_t)((a.c.cap + per - 1) / per) * a.c.B * a.c.Hkv)), kMassThreads, 0, 1, s, a, p.sp,
                         unit_rows);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace attn
