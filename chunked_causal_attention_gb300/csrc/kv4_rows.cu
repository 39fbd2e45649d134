// Rows of the 4-bit cache: quantise and store, load and dequantise.
//
// Both are bound by memory: a row of D dims is 2D bytes of bf16 on one side and
// D/2 + D/16 on the other. Two adjacent lanes share a block of 16 dims; each
// holds 8 (one 16-byte bf16 access, one 4-byte code access) and they exchange
// the block's maximum with one shuffle.
//
// Quantising: s = e4m3(max / (6 ts)) by one IEEE division a block, so a maximum
// that lies between two scales rounds to even as its exact quotient does. The
// codes need x / d with d = s ts only as far as rounding to e2m1 sees it: the
// borders between codes are multiples of 1/4. x has 8 significant bits, d at most
// 4, and a quotient that is not on a border t is at least 2^-11 off it (x - t d is
// a whole multiple of the smaller unit of x and t d), so x * (1/d), which is
// within 2^-21, only has to be pulled onto a border when it is on one: adding and
// taking away 48 rounds it to a multiple of 2^-18.
#include <algorithm>

#include "kv4_device.cuh"

namespace attn {
namespace {

using namespace kv4;

constexpr int kThreads = 256;

// Row r of the call: which sequence and head, the offset of its bf16 row, its cache row. False: skipped.
__device__ __forceinline__ bool locate(const Kv4RowsArgs& a, uint32_t r, int64_t& off, int64_t& row) {
    int32_t b, h, t;
    int64_t slot;
    if (a.cu) {
        // packed: r = token * Hkv + head; the sequence is the last one that starts at or before the token
        const uint32_t tok = a.by_h.div(r);
        h = (int32_t)(r - tok * a.by_h.d);
        int32_t lo = 0, hi = a.c.B;            // cu[lo] <= tok < cu[hi] where the offsets are in order
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) >> 1;
            if (a.cu[mid] <= (int32_t)tok) lo = mid; else hi = mid;
        }
        b = lo;
        t = (int32_t)tok - a.cu[b];
        off = (int64_t)tok * a.st + (int64_t)h * a.sh;
        slot = (int32_t)tok < a.cu[b + 1] && t >= 0 ? (int64_t)a.pos[b] + t : -1;
    } else {
        const uint32_t bh = a.by_t.div(r);
        t = (int32_t)(r - bh * a.by_t.d);
        b = (int32_t)a.by_h.div(bh);
        h = (int32_t)(bh - (uint32_t)b * a.by_h.d);
        off = (int64_t)b * a.sb + (int64_t)h * a.sh + (int64_t)t * a.st;
        slot = (int64_t)a.pos[b] + t;
    }
    if (slot < 0 || slot >= a.c.cap) return false;
    row = (int64_t)b * a.c.sb + (int64_t)h * a.c.sh + slot;
    return true;
}

// blockIdx.y: 0 keys, 1 values. Thread = (row of the block's group, 8 dims); a
// row takes 2 * nb threads, so the two of a block of 16 dims are adjacent lanes.
template <bool STORE>
__global__ void __launch_bounds__(kThreads) kv4_rows_kernel(const Kv4RowsArgs a, int32_t rows_per_block) {
    const int per = 2 * a.c.nb;
    const int r0 = threadIdx.x / per, part = threadIdx.x - r0 * per;
    const bool on = r0 < rows_per_block && part * 8 < a.c.D;     // lanes past D help their neighbour's shuffle only
    const bool val = blockIdx.y != 0;
    uint8_t* codes = val ? a.c.vc : a.c.kc;
    uint8_t* scales = val ? a.c.vs : a.c.ks;
    const float ts = val ? a.c.v_scale : a.c.k_scale;
    __nv_bfloat16* x = reinterpret_cast<__nv_bfloat16*>(val ? a.v : a.k);
    const int64_t step = (int64_t)gridDim.x * rows_per_block;
    for (int64_t base = (int64_t)blockIdx.x * rows_per_block; base < a.rows; base += step) {
        const int64_t r = base + r0;
        int64_t off = 0, row = 0;
        bool live = on && r < a.rows;
        if (live && !locate(a, (uint32_t)r, off, row)) {
            live = false;
            set_error(a.status, ATTN_E_BOUNDS);
        }
        if constexpr (STORE) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live) w = *reinterpret_cast<const uint4*>(x + off + part * 8);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            // |x| as bf16 bits orders like the values, infinities and NaN last
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max(top, max(u[i] & 0x7FFFu, (u[i] >> 16) & 0x7FFFu));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            const float amax = __uint_as_float(top << 16);
            const uint32_t s8 = top >= 0x7F80u ? 0x7Fu : e4m3(__fdiv_rn(amax, 6.f * ts));
            const float s = __half2float(__low2half(as_half2(scales_f16x2(s8))));
            const float d = s * ts;
            const float inv = s > 0.f ? __frcp_rn(d) : 0.f;     // 0 and NaN scales: codes 0
            uint32_t c = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lo = __uint_as_float(u[i] << 16), hi = __uint_as_float(u[i] & 0xFFFF0000u);
                // to a multiple of 2^-18, the sign of zero kept
                const float y0 = copysignf((fabsf(lo) * inv + 48.f) - 48.f, lo);
                const float y1 = copysignf((fabsf(hi) * inv + 48.f) - 48.f, hi);
                c |= e2m1x2(y0, y1) << (8 * i);
            }
            if (s8 == 0x7Fu) c = 0;
            if (live) {
                *reinterpret_cast<uint32_t*>(codes + row * a.c.cb + part * 4) = c;
                if (!(part & 1)) scales[row * a.c.nb + (part >> 1)] = (uint8_t)s8;
            }
        } else if (live) {
            const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + row * a.c.cb + part * 4);
            const uint32_t s8 = scales[row * a.c.nb + (part >> 1)];
            const float d = __half2float(__low2half(as_half2(scales_f16x2(s8)))) * ts;
            const uint32_t f[4] = {codes_f16x2<0>(c), codes_f16x2<1>(c), codes_f16x2<2>(c), codes_f16x2<3>(c)};
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 y = __half22float2(as_half2(f[i]));
                u[i] = pack_bf16(y.x * d, y.y * d);
            }
            *reinterpret_cast<uint4*>(x + off + part * 8) = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
}

template <bool STORE>
cudaError_t launch(const Kv4RowsArgs& a, cudaStream_t s) {
    const int rows_per_block = kThreads / (2 * a.c.nb);
    const int64_t blocks = (a.rows + rows_per_block - 1) / rows_per_block;
    const dim3 grid((unsigned)std::min<int64_t>(blocks, (int64_t)device_sm_count() * 16), 2);
    kv4_rows_kernel<STORE><<<grid, kThreads, 0, s>>>(a, rows_per_block);
    return counted(cudaGetLastError());
}

}  // namespace

cudaError_t launch_kv4_store(const Kv4RowsArgs& a, cudaStream_t s) { return launch<true>(a, s); }
cudaError_t launch_kv4_load(const Kv4RowsArgs& a, cudaStream_t s) { return launch<false>(a, s); }

}  // namespace attn
