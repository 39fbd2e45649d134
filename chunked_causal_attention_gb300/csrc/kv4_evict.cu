// Eviction by accumulated attention weight: choose the slots, then move them.
//
// Choosing is a radix selection: the masses map to 32-bit keys that order as they
// do, and four histograms of eight bits each narrow down the value of the last
// slot that is kept; a second pass counts the slots above it and the ties, of
// which the lowest are kept, and writes the slots in order. One block per
// (sequence, key/value head).
#include <algorithm>

#include "kv4_device.cuh"

namespace attn {
namespace {

using namespace kv4;

constexpr int kThreads = 1024;

// Orders as the masses do: NaN above everything, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum of x over the block and the block's total.
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
    uint32_t before = 0;
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
    __syncthreads();
    return before + y - x;
}

__global__ void __launch_bounds__(kThreads) choose_kernel(const Kv4EvictArgs a) {
    const int bh = blockIdx.x, b = bh / a.src.Hkv;
    const int n = length_of(a.lens, b, (int32_t)min((int64_t)a.src.cap, a.mass_ld), a.status);
    const int m = min(n, a.keep), recent = min(m, a.recent);
    const int cand = n - recent, want = m - recent;       // choose `want` of the slots [0, cand)
    const float* mass = a.mass + (int64_t)bh * a.mass_ld;
    int32_t* out = a.slots + (int64_t)bh * a.keep;
    __shared__ uint32_t hist[256], warp_sums[kThreads / 32], sh_prefix, sh_left;
    uint32_t prefix = 0, left = want;                     // key of the last kept slot; how many of it and below its prefix
    if (want < cand && want > 0) {
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            for (int i = threadIdx.x; i < 256; i += kThreads) hist[i] = 0;
            __syncthreads();
            for (int j = threadIdx.x; j < cand; j += kThreads) {
                const uint32_t u = order_key(mass[j]);
                if (pass == 0 || (u >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(u >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                uint32_t above = 0;
                int d = 255;
                while (d > 0 && above + hist[d] < left) above += hist[d--];
                sh_prefix = prefix | ((uint32_t)d << shift);
                sh_left = left - above;
            }
            __syncthreads();
            prefix = sh_prefix;
            left = sh_left;
        }
    }
    // kept: keys above `prefix`, and the first `left` of those equal to it
    uint32_t base = 0, ties = 0;
    if (want >= cand) {
        for (int j = threadIdx.x; j < cand; j += kThreads) out[j] = j;
    } else if (want > 0) {
        for (int j0 = 0; j0 < cand; j0 += kThreads) {
            const int j = j0 + threadIdx.x;
            const uint32_t u = j < cand ? order_key(mass[j]) : 0u;
            const bool eq = j < cand && u == prefix;
            uint32_t tile_ties, tile_kept;
            const uint32_t rank = ties + block_scan(eq, warp_sums, tile_ties);
            const bool kept = (j < cand && u > prefix) || (eq && rank < left);
            const uint32_t at = base + block_scan(kept, warp_sums, tile_kept);
            if (kept && at < (uint32_t)want) out[at] = j;
            ties += tile_ties;
            base += tile_kept;
        }
    }
    for (int i = threadIdx.x; i < recent; i += kThreads) out[want + i] = cand + i;
    for (int i = m + threadIdx.x; i < a.keep; i += kThreads) out[i] = -1;
}

// One warp per kept row: its codes, scales and mass. Block (0, 0) writes the lengths.
__global__ void __launch_bounds__(256) move_kernel(const Kv4EvictArgs a) {
    const int chunks = (a.keep + 7) / 8, bh = blockIdx.x / chunks, chunk = blockIdx.x - bh * chunks;
    const int b = bh / a.src.Hkv, h = bh % a.src.Hkv, lane = threadIdx.x & 31;
    if (chunk == 0 && h == 0 && threadIdx.x == 0) {
        const int n = min(max(a.lens[b], 0), (int)min((int64_t)a.src.cap, a.mass_ld));
        a.lens_out[b] = min(n, a.keep);
    }
    const int i = chunk * 8 + (threadIdx.x >> 5);
    if (i >= a.keep) return;
    const int j = a.slots[(int64_t)bh * a.keep + i];
    if (j < 0 || j >= a.src.cap) return;
    const int64_t from = (int64_t)b * a.src.sb + (int64_t)h * a.src.sh + j;
    const int64_t to = (int64_t)b * a.dst.sb + (int64_t)h * a.dst.sh + i;
    for (int w = lane; w < a.src.cb / 4; w += 32) {
        reinterpret_cast<uint32_t*>(a.dst.kc + to * a.dst.cb)[w] = reinterpret_cast<const uint32_t*>(a.src.kc + from * a.src.cb)[w];
        reinterpret_cast<uint32_t*>(a.dst.vc + to * a.dst.cb)[w] = reinterpret_cast<const uint32_t*>(a.src.vc + from * a.src.cb)[w];
    }
    if (lane < a.src.nb) {
        a.dst.ks[to * a.dst.nb + lane] = a.src.ks[from * a.src.nb + lane];
        a.dst.vs[to * a.dst.nb + lane] = a.src.vs[from * a.src.nb + lane];
    }
    if (lane == 0 && a.mass_out) a.mass_out[(int64_t)bh * a.mass_out_ld + i] = a.mass[(int64_t)bh * a.mass_ld + j];
}

}  // namespace

cudaError_t launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t s) {
    const int BH = a.src.B * a.src.Hkv;
    choose_kernel<<<BH, kThreads, 0, s>>>(a);
    cudaError_t e = counted(cudaGetLastError());
    if (e != cudaSuccess) return e;
    move_kernel<<<(unsigned)((int64_t)((a.keep + 7) / 8) * BH), 256, 0, s>>>(a);
    return counted(cudaGetLastError());
}

}  // namespace attn
