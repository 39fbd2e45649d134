// Eviction by accumulated attention weight: choose the slots, then move them.
//
// Choosing is a radix selection: the masses map to 32-bit keys that order as they
// do, and four histograms of eight bits each narrow down the key of the last slot
// that is kept; then the slots above it and the first of those equal to it are
// written in order. A cluster of up to eight blocks shares a (sequence, key/value
// head): each holds a stretch of the masses, read from memory once, as keys in its
// shared memory; every block reads the others' histograms and comes to the same
// digit, so a pass costs one cluster barrier.
//
// Moving is bound by the latency of two dependent reads (slot, row) and by bytes: a
// thread takes one 16-byte piece of a row, of four rows at a time.
//
// Measured: 131072 masses of 8 heads to 4096 slots 25 us (choosing 19), 48 x 8 heads of
// 2176 slots to 2048 64 us (choosing 14; moving 226 MB 50, with one piece of one row at a
// time 95), 1M masses of 8 heads 151 us.
#include <algorithm>

#include "kv4_device.cuh"

namespace attn {
namespace {

using namespace kv4;

constexpr int kPer = 4;                        // neighbouring masses of a thread and tile
constexpr int kMaxCluster = 8;
constexpr int kHeld = 32768;                   // keys that a block keeps in shared memory; the others it reads again

// Orders as the masses do: NaN above everything, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// A 32-bit word of block `rank`'s shared memory, at the address of this block's `p`.
__device__ __forceinline__ uint32_t cluster_load(const uint32_t* p, uint32_t rank) {
    uint32_t a = smem_u32(p), v;
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;\n" : "+r"(a) : "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// Exclusive prefix sum of x over the block, and the block's sum.
template <int THREADS>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* warp_sums, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t y = x;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const uint32_t z = __shfl_up_sync(0xffffffffu, y, m);
        if (lane >= m) y += z;
    }
    if (lane == 31) warp_sums[warp] = y;
    __syncthreads();
    const uint32_t w = lane < THREADS / 32 ? warp_sums[lane] : 0u;
    uint32_t v = w;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const uint32_t z = __shfl_up_sync(0xffffffffu, v, m);
        if (lane >= m) v += z;
    }
    total = __shfl_sync(0xffffffffu, v, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, v - w, warp);
    __syncthreads();
    return before + y - x;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) choose_kernel(const Kv4EvictArgs a, const int32_t blocks) {
    constexpr int kChunk = THREADS * kPer, kHeldTiles = kHeld / kChunk;
    extern __shared__ __align__(16) uint32_t held[];     // keys of the first kHeldTiles tiles
    __shared__ uint32_t hist[2][256], warp_sums[32], found[2], counts[2];
    const int rank = (int)cluster_rank(), bh = blockIdx.x / blocks, b = bh / a.src.Hkv, tid = threadIdx.x;
    grid_wait();
    grid_go();
    const int n = length_of(a.lens, b, (int32_t)min((int64_t)a.src.cap, a.mass_ld), a.status);
    const int m = min(n, a.keep), recent = min(m, a.recent);
    const int cand = n - recent, want = m - recent;      // choose `want` of the slots [0, cand)
    const float* mass = a.mass + (int64_t)bh * a.mass_ld;
    int32_t* out = a.slots + (int64_t)bh * a.keep;
    const bool choose = want > 0 && want < cand;         // the same for every block of the cluster
    // this block's stretch: whole tiles
    const int tiles = (cand + kChunk - 1) / kChunk, per = (tiles + blocks - 1) / blocks;
    const int first = min(rank * per, tiles), last = min(first + per, tiles);
    if (choose) {
        auto keys = [&](int tile, uint32_t (&u)[kPer]) {
            if (tile - first < kHeldTiles) {
                const uint4 x = *reinterpret_cast<const uint4*>(held + (tile - first) * kChunk + tid * kPer);
                u[0] = x.x; u[1] = x.y; u[2] = x.z; u[3] = x.w;
            } else {
                const int j = tile * kChunk + tid * kPer;
#pragma unroll
                for (int i = 0; i < kPer; ++i) u[i] = j + i < cand ? order_key(mass[j + i]) : 0u;
            }
        };
        uint32_t prefix = 0, left = want;                // key of the last kept slot; slots still to choose with its prefix
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            uint32_t* h = hist[pass & 1];
            if (tid < 256) h[tid] = 0;
            __syncthreads();
            for (int tile = first; tile < last; ++tile) {
                uint32_t u[kPer];
                const int j = tile * kChunk + tid * kPer;
                if (pass == 0) {
#pragma unroll
                    for (int i = 0; i < kPer; ++i) u[i] = j + i < cand ? order_key(mass[j + i]) : 0u;
                    if (tile - first < kHeldTiles)
                        *reinterpret_cast<uint4*>(held + (tile - first) * kChunk + tid * kPer) = make_uint4(u[0], u[1], u[2], u[3]);
                } else {
                    keys(tile, u);
                }
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (j + i < cand && (pass == 0 || (u[i] >> (shift + 8)) == (prefix >> (shift + 8))))
                        atomicAdd(&h[(u[i] >> shift) & 255u], 1u);
            }
            cluster_sync();
            if (tid < 256) {
                uint32_t x = 0, v[kMaxCluster];
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r) v[r] = r < blocks ? cluster_load(h + tid, r) : 0u;
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r) x += v[r];
                // slots with a digit above this one, by a scan from the top
                uint32_t y = x;
                const int lane = tid & 31;
#pragma unroll
                for (int s = 1; s < 32; s <<= 1) {
                    const uint32_t z = __shfl_down_sync(0xffffffffu, y, s);
                    if (lane + s < 32) y += z;
                }
                if (lane == 0) warp_sums[tid >> 5] = y;
                asm volatile("bar.sync 1, 256;\n" ::: "memory");
                for (int w = (tid >> 5) + 1; w < 8; ++w) y += warp_sums[w];
                if (y >= left && y - x < left) {
                    found[0] = prefix | ((uint32_t)tid << shift);
                    found[1] = left - (y - x);
                }
            }
            __syncthreads();
            prefix = found[0];
            left = found[1];
        }
        // how many of this block are above the key and equal to it, and of the blocks before
        uint32_t above = 0, equal = 0;
        for (int tile = first; tile < last; ++tile) {
            uint32_t u[kPer];
            keys(tile, u);
            const int j = tile * kChunk + tid * kPer;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                above += j + i < cand && u[i] > prefix;
                equal += j + i < cand && u[i] == prefix;
            }
        }
        uint32_t t_above, t_equal;
        block_scan<THREADS>(above, warp_sums, t_above);
        block_scan<THREADS>(equal, warp_sums, t_equal);
        if (tid == 0) {
            counts[0] = t_above;
            counts[1] = t_equal;
        }
        cluster_sync();
        uint32_t base = 0, ties = 0;
        for (int r = 0; r < rank; ++r) {
            base += cluster_load(&counts[0], r);
            ties += cluster_load(&counts[1], r);
        }
        base += min(ties, left);                         // of the ties before, the first `left` are kept
        for (int tile = first; tile < last; ++tile) {
            uint32_t u[kPer];
            keys(tile, u);
            const int j = tile * kChunk + tid * kPer;
            uint32_t eq = 0, tot;
#pragma unroll
            for (int i = 0; i < kPer; ++i) eq += j + i < cand && u[i] == prefix;
            uint32_t rank_eq = ties + block_scan<THREADS>(eq, warp_sums, tot);
            ties += tot;
            uint32_t kept = 0;
            bool k[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const bool in = j + i < cand, e = in && u[i] == prefix;
                k[i] = in && (u[i] > prefix || (e && rank_eq < left));
                rank_eq += e;
                kept += k[i];
            }
            uint32_t at = base + block_scan<THREADS>(kept, warp_sums, tot);
            base += tot;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (k[i] && at < (uint32_t)want) out[at++] = j + i;
        }
        cluster_sync();                                  // no block leaves while another may read its shared memory
    } else if (want > 0) {
        for (int j = rank * THREADS + tid; j < cand; j += blocks * THREADS) out[j] = j;
    }
    for (int i = rank * THREADS + tid; i < recent; i += blocks * THREADS) out[want + i] = cand + i;
    for (int i = m + rank * THREADS + tid; i < a.keep; i += blocks * THREADS) out[i] = -1;
}

// The kept rows' codes, scales and masses. A thread takes one piece (CB bytes of codes,
// SB of scales, or the mass) of kMoves rows at a time, so that the two reads that depend
// on each other (slot, piece) are in flight for several rows.
constexpr int kMoves = 4;
constexpr int kMoveThreads = 256;
template <int CB, int SB>
__global__ void __launch_bounds__(kMoveThreads)
    move_kernel(const Kv4EvictArgs a, const int32_t pieces, const FastDiv by_keep, const FastDiv by_h) {
    const int nc = a.src.cb / CB, ns = a.src.nb / SB, rows_per_block = kMoveThreads / pieces;
    const int r0 = threadIdx.x / pieces;
    int p = threadIdx.x - r0 * pieces;
    const uint8_t* src;
    uint8_t* dst;
    int pitch, bytes;
    int64_t fb = a.src.sb, fh = a.src.sh, tb = a.dst.sb, th = a.dst.sh;   // rows from and to, of a sequence and a head
    if (p < 2 * nc) {
        const bool v = p >= nc;
        p -= v ? nc : 0;
        src = (v ? a.src.vc : a.src.kc) + p * CB;
        dst = (v ? a.dst.vc : a.dst.kc) + p * CB;
        pitch = a.src.cb;
        bytes = CB;
    } else if (p < 2 * (nc + ns)) {
        p -= 2 * nc;
        const bool v = p >= ns;
        p -= v ? ns : 0;
        src = (v ? a.src.vs : a.src.ks) + p * SB;
        dst = (v ? a.dst.vs : a.dst.ks) + p * SB;
        pitch = a.src.nb;
        bytes = SB;
    } else {
        src = reinterpret_cast<const uint8_t*>(a.mass);
        dst = reinterpret_cast<uint8_t*>(a.mass_out);
        pitch = bytes = 4;
        fb = a.mass_ld * a.src.Hkv;
        fh = a.mass_ld;
        tb = a.mass_out_ld * a.src.Hkv;
        th = a.mass_out_ld;
    }
    grid_wait();                                         // the slots
    grid_go();
    const int64_t rows = (int64_t)a.src.B * a.src.Hkv * a.keep, step = (int64_t)gridDim.x * rows_per_block;
    for (int64_t base = (int64_t)blockIdx.x * rows_per_block + r0; r0 < rows_per_block && base < rows; base += step * kMoves) {
        int32_t j[kMoves];
#pragma unroll
        for (int x = 0; x < kMoves; ++x) j[x] = base + x * step < rows ? a.slots[base + x * step] : -1;
        int64_t to[kMoves];
        uint4 v[kMoves];
#pragma unroll
        for (int x = 0; x < kMoves; ++x) {
            if (j[x] < 0 || j[x] >= a.src.cap) continue;
            const uint32_t r = (uint32_t)(base + x * step), bh = by_keep.div(r), b = by_h.div(bh);
            const int32_t i = (int32_t)(r - bh * by_keep.d), h = (int32_t)(bh - b * by_h.d);
            const uint8_t* f = src + (b * fb + h * fh + j[x]) * pitch;
            to[x] = (b * tb + h * th + i) * pitch;
            if (bytes == 16) v[x] = *reinterpret_cast<const uint4*>(f);
            else if (bytes == 8) *reinterpret_cast<uint2*>(&v[x]) = *reinterpret_cast<const uint2*>(f);
            else if (bytes == 4) v[x].x = *reinterpret_cast<const uint32_t*>(f);
            else v[x].x = *f;
        }
#pragma unroll
        for (int x = 0; x < kMoves; ++x) {
            if (j[x] < 0 || j[x] >= a.src.cap) continue;
            uint8_t* t = dst + to[x];
            if (bytes == 16) *reinterpret_cast<uint4*>(t) = v[x];
            else if (bytes == 8) *reinterpret_cast<uint2*>(t) = make_uint2(v[x].x, v[x].y);
            else if (bytes == 4) *reinterpret_cast<uint32_t*>(t) = v[x].x;
            else *t = (uint8_t)v[x].x;
        }
    }
    // lens_out may be lens: every block of the kernel before has read it by now, and this block alone does here
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.src.B; b += kMoveThreads) {
            const int n = min(max(a.lens[b], 0), (int)min((int64_t)a.src.cap, a.mass_ld));
            a.lens_out[b] = min(n, a.keep);
        }
}

template <int CB, int SB>
cudaError_t launch_move(const Kv4EvictArgs& a, cudaStream_t s) {
    const int pieces = 2 * (a.src.cb / CB + a.src.nb / SB) + (a.mass_out ? 1 : 0);
    const int64_t rows = (int64_t)a.src.B * a.src.Hkv * a.keep, per = kMoveThreads / pieces;
    return launch_early(move_kernel<CB, SB>, dim3((unsigned)std::min<int64_t>((rows + per - 1) / per, (int64_t)device_sm_count() * 8)),
                        kMoveThreads, 0, 1, s, a, (int32_t)pieces, FastDiv::of((uint32_t)a.keep),
                        FastDiv::of((uint32_t)a.src.Hkv));
}

template <int THREADS>
cudaError_t launch_choose(const Kv4EvictArgs& a, cudaStream_t s) {
    constexpr int kChunk = THREADS * kPer;
    const int64_t BH = (int64_t)a.src.B * a.src.Hkv;
    // blocks of a cluster: a power of two, no more than there are tiles in the cache
    int blocks = 1;
    while (blocks < kMaxCluster && (int64_t)blocks * kChunk < a.src.cap) blocks *= 2;
    // enough blocks for every SM without them: one a head
    if (BH >= 2 * device_sm_count()) blocks = 1;
    const int tiles = (a.src.cap + kChunk - 1) / kChunk;
    const int smem = std::min((tiles + blocks - 1) / blocks * kChunk, kHeld) * 4;
    if (smem > 40 * 1024) {                      // 48 KB with the static part is what a block may have without asking
        // always the most that any call takes: the limit is the function's, and a call of another thread may be
        // between its own limit and its launch
        const cudaError_t e = cudaFuncSetAttribute(choose_kernel<THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld * 4);
        if (e != cudaSuccess) return e;
    }
    return launch_early(choose_kernel<THREADS>, dim3((unsigned)(BH * blocks)), THREADS, smem, blocks, s, a, (int32_t)blocks);
}

}  // namespace

cudaError_t launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t s) {
    // many heads: smaller blocks, more of them on an SM at once
    cudaError_t e = (int64_t)a.src.B * a.src.Hkv >= 2 * device_sm_count() ? launch_choose<512>(a, s) : launch_choose<1024>(a, s);
    if (e != cudaSuccess) return e;
    const bool wide = a.src.cb % 16 == 0, scales = a.src.nb % 8 == 0;
    return wide ? (scales ? launch_move<16, 8>(a, s) : launch_move<16, 1>(a, s))
                : (scales ? launch_move<4, 8>(a, s) : launch_move<4, 1>(a, s));
}

}  // namespace attn
