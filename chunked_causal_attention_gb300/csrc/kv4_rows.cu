// Rows of the 4-bit cache: quantise and store, load and dequantise.
//
// Both are bound by memory: a row of D dims is 2D bytes of bf16 on one side and
// D/2 + D/16 on the other. A thread takes a block of 16 dims (two 16-byte accesses
// of bf16, one of 8 bytes of codes, one scale) of two rows at a time, so that its
// loads are in flight together.
//
// Measured, 16384 rows of 32 heads of 128 dims, keys and values: store 68 us (5.0 TB/s;
// its issue slots are 80% busy, 254 instructions for a block of 16), load 66 us (5.2 TB/s,
// four fifths of it writes). With 8 dims a thread and one row at a time 108 and 71 us.
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
#include "tc_common.cuh"

namespace attn {
namespace {

using namespace kv4;

constexpr int kThreads = 256;
constexpr int kAtOnce = 2;      // rows of a thread in flight

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

// |x| of two bf16, the larger of each half: as bits they order like the values, infinities and NaN last.
__device__ __forceinline__ uint32_t larger2(uint32_t top, uint32_t u) { return __vmaxu2(top, u & 0x7FFF7FFFu); }

// Eight values (four words of bf16) to four bytes of codes, inv = 1 / d.
__device__ __forceinline__ uint32_t codes8(const uint4& w, float inv) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(u[i] << 16), hi = __uint_as_float(u[i] & 0xFFFF0000u);
        // |x| / d to a multiple of 2^-18, the sign of zero kept
        const float2 y = tc::fadd2(tc::ffma2(make_float2(fabsf(lo), fabsf(hi)), make_float2(inv, inv), make_float2(48.f, 48.f)),
                                   make_float2(-48.f, -48.f));
        c |= e2m1x2(copysignf(y.x, lo), copysignf(y.y, hi)) << (8 * i);
    }
    return c;
}

// Four bytes of codes to eight values times d.
__device__ __forceinline__ uint4 values8(uint32_t c, float d) {
    const uint32_t f[4] = {codes_f16x2<0>(c), codes_f16x2<1>(c), codes_f16x2<2>(c), codes_f16x2<3>(c)};
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = __half22float2(as_half2(f[i]));
        u[i] = pack_bf16(y.x * d, y.y * d);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// blockIdx.y: 0 keys, 1 values. A thread is (row of the block's group, block of 16 dims).
template <bool STORE>
__global__ void __launch_bounds__(kThreads) kv4_rows_kernel(const Kv4RowsArgs a, int32_t rows_per_block) {
    grid_wait();
    grid_go();
    const int per = a.c.nb;
    const int r0 = threadIdx.x / per, part = threadIdx.x - r0 * per;
    if (r0 >= rows_per_block) return;
    const bool second = part * 16 + 8 < a.c.D;           // D need not be a multiple of 16
    const bool val = blockIdx.y != 0;
    uint8_t* codes = val ? a.c.vc : a.c.kc;
    uint8_t* scales = val ? a.c.vs : a.c.ks;
    const float ts = val ? a.c.v_scale : a.c.k_scale;
    __nv_bfloat16* x = reinterpret_cast<__nv_bfloat16*>(val ? a.v : a.k) + part * 16;
    const int64_t step = (int64_t)gridDim.x * rows_per_block * kAtOnce;
    for (int64_t base = (int64_t)blockIdx.x * rows_per_block * kAtOnce; base < a.rows; base += step) {
        int64_t off[kAtOnce], row[kAtOnce];
        bool live[kAtOnce];
        uint4 w[kAtOnce][2];
        uint2 c[kAtOnce];
        uint32_t s8[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int64_t r = base + i * rows_per_block + r0;
            live[i] = r < a.rows;
            off[i] = row[i] = 0;
            if (live[i] && !locate(a, (uint32_t)r, off[i], row[i])) {
                live[i] = false;
                set_error(a.status, ATTN_E_BOUNDS);
            }
            w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
            c[i] = make_uint2(0, 0);
            s8[i] = 0;
            if (live[i]) {
                if constexpr (STORE) {
                    w[i][0] = *reinterpret_cast<const uint4*>(x + off[i]);
                    if (second) w[i][1] = *reinterpret_cast<const uint4*>(x + off[i] + 8);
                } else {
                    const uint8_t* p = codes + row[i] * a.c.cb + part * 8;
                    c[i].x = *reinterpret_cast<const uint32_t*>(p);       // rows start at multiples of 4 bytes
                    if (second) c[i].y = *reinterpret_cast<const uint32_t*>(p + 4);
                    s8[i] = scales[row[i] * a.c.nb + part];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if (!live[i]) continue;
            if constexpr (STORE) {
                const uint4 p = w[i][0], q = w[i][1];
                uint32_t top = larger2(larger2(larger2(larger2(0u, p.x), p.y), p.z), p.w);
                top = larger2(larger2(larger2(larger2(top, q.x), q.y), q.z), q.w);
                top = max(top & 0xFFFFu, top >> 16);
                const uint32_t s = top >= 0x7F80u ? 0x7Fu : e4m3(__fdiv_rn(__uint_as_float(top << 16), 6.f * ts));
                const float f = __half2float(__low2half(as_half2(scales_f16x2(s))));
                // 0 and NaN scales: codes 0
                const float inv = f > 0.f ? __frcp_rn(f * ts) : 0.f;
                uint32_t c0 = codes8(p, inv), c1 = codes8(q, inv);
                if (s == 0x7Fu) c0 = c1 = 0;
                uint8_t* d = codes + row[i] * a.c.cb + part * 8;
                if (second && (a.c.cb & 7) == 0) {
                    *reinterpret_cast<uint2*>(d) = make_uint2(c0, c1);
                } else {
                    *reinterpret_cast<uint32_t*>(d) = c0;
                    if (second) *reinterpret_cast<uint32_t*>(d + 4) = c1;
                }
                scales[row[i] * a.c.nb + part] = (uint8_t)s;
            } else {
                const float d = __half2float(__low2half(as_half2(scales_f16x2(s8[i])))) * ts;
                *reinterpret_cast<uint4*>(x + off[i]) = values8(c[i].x, d);
                if (second) *reinterpret_cast<uint4*>(x + off[i] + 8) = values8(c[i].y, d);
            }
        }
    }
}

template <bool STORE>
cudaError_t launch(const Kv4RowsArgs& a, cudaStream_t s) {
    const int rows_per_block = kThreads / a.c.nb;
    const int64_t blocks = (a.rows + rows_per_block * kAtOnce - 1) / (rows_per_block * kAtOnce);
    // measured on 16K rows of 32 heads of 128 dims: the store 68 us with up to 16 blocks an SM and tensor
    // (72 with 64), the load 66 with 64 (70 with 16, 74 with 8)
    const dim3 grid((unsigned)std::min<int64_t>(blocks, (int64_t)device_sm_count() * (STORE ? 16 : 64)), 2);
    return launch_early(kv4_rows_kernel<STORE>, grid, kThreads, 0, 1, s, a, (int32_t)rows_per_block);
}

}  // namespace

cudaError_t launch_kv4_store(const Kv4RowsArgs& a, cudaStream_t s) { return launch<true>(a, s); }
cudaError_t launch_kv4_load(const Kv4RowsArgs& a, cudaStream_t s) { return launch<false>(a, s); }

}  // namespace attn
