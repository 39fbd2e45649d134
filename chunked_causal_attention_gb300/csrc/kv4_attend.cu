// Attention of the newest tokens over the 4-bit cache: the simple form. One
// block per query row, four warps over its keys with a running maximum and sum,
// lanes over dims; the slots' weights by a second pass over the keys.
#include "kv4_device.cuh"

namespace attn {
namespace {

using namespace kv4;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// This lane's 8 dims of a cached row.
__device__ __forceinline__ void row8(const uint8_t* codes, const uint8_t* scales, float ts, int lane, bool on,
                                     float (&x)[8]) {
    const uint32_t c = on ? *reinterpret_cast<const uint32_t*>(codes + lane * 4) : 0u;
    const uint32_t s = on ? scales[lane >> 1] : 0u;
    const float d = __half2float(__low2half(as_half2(scales_f16x2(s)))) * ts;
    const uint32_t f[4] = {codes_f16x2<0>(c), codes_f16x2<1>(c), codes_f16x2<2>(c), codes_f16x2<3>(c)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = __half22float2(as_half2(f[i]));
        x[2 * i] = y.x * d;
        x[2 * i + 1] = y.y * d;
    }
}

__device__ __forceinline__ void query8(const Kv4AttendArgs& a, int b, int h, int i, int lane, bool on, float (&q)[8]) {
    const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(a.q) + (int64_t)b * a.g.sb + (int64_t)h * a.g.sh +
                             (int64_t)i * a.g.st;
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = on ? __bfloat162float(p[lane * 8 + j]) : 0.f;
}

__global__ void __launch_bounds__(128) attend_rows(const Kv4AttendArgs a) {
    const int r = blockIdx.x;                       // (b, h, i)
    const int i = r % a.g.T, h = r / a.g.T % a.g.H, b = r / a.g.T / a.g.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool on = lane * 8 < a.c.D;
    const int hk = h / (a.g.H / a.g.Hkv);
    const int64_t most = a.mass_out && a.mass_ld < a.c.cap ? a.mass_ld : a.c.cap;
    const int n = length_of(a.lens, b, (int32_t)most, a.status);
    const int seen = n - a.g.T + i + 1;             // slots [0, seen)
    float q[8], o[8] = {}, m = -INFINITY, l = 0.f;
    query8(a, b, h, i, lane, on, q);
    const int64_t row0 = (int64_t)b * a.c.sb + (int64_t)hk * a.c.sh;
    for (int j = warp; j < seen; j += 4) {
        float x[8];
        row8(a.c.kc + (row0 + j) * a.c.cb, a.c.ks + (row0 + j) * a.c.nb, a.c.k_scale, lane, on, x);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(q[e], x[e], s);
        s = warp_sum(s) * a.g.scale;
        const float mn = s > m ? s : m;
        const float w = expf(m - mn), p = expf(s - mn);
        row8(a.c.vc + (row0 + j) * a.c.cb, a.c.vs + (row0 + j) * a.c.nb, a.c.v_scale, lane, on, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(o[e], w, p * x[e]);
        l = fmaf(l, w, p);
        m = mn;
    }
    __shared__ float so[4][256], sm[4], sl[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) so[warp][lane * 8 + e] = o[e];
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
    __syncthreads();
    float top = -INFINITY;
    for (int w = 0; w < 4; ++w) top = sl[w] != 0.f && !(sm[w] <= top) ? sm[w] : top;
    float total = 0.f, f[4];
    for (int w = 0; w < 4; ++w) {
        f[w] = sl[w] != 0.f ? expf(sm[w] - top) : 0.f;
        total += f[w] * sl[w];
    }
    const bool none = seen <= 0;
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.o) + (int64_t)b * a.g.sb + (int64_t)h * a.g.sh +
                         (int64_t)i * a.g.st;
    for (int d = threadIdx.x; d < a.c.D; d += 128) {
        float y = 0.f;
        for (int w = 0; w < 4; ++w) y += sl[w] != 0.f ? f[w] * so[w][d] : 0.f;
        out[d] = __float2bfloat16(none ? 0.f : y / total);
    }
    if (threadIdx.x == 0) a.lse[r] = none ? -INFINITY : top + logf(total);
}

// One warp per slot: its weight over the rows of its key/value head.
__global__ void __launch_bounds__(256) attend_mass(const Kv4AttendArgs a) {
    const int lane = threadIdx.x & 31;
    const int j = blockIdx.x * 8 + (threadIdx.x >> 5), bh = blockIdx.y;
    const int b = bh / a.c.Hkv, hk = bh % a.c.Hkv, G = a.g.H / a.c.Hkv;
    const int n = length_of(a.lens, b, (int32_t)min((int64_t)a.c.cap, a.mass_ld), a.status);
    if (j >= n) return;
    const bool on = lane * 8 < a.c.D;
    const int64_t row = (int64_t)b * a.c.sb + (int64_t)hk * a.c.sh + j;
    float x[8], w = 0.f;
    row8(a.c.kc + row * a.c.cb, a.c.ks + row * a.c.nb, a.c.k_scale, lane, on, x);
    for (int h = hk * G; h < hk * G + G; ++h)
        for (int i = 0; i < a.g.T; ++i) {
            if (j > n - a.g.T + i) continue;
            float q[8], s = 0.f;
            query8(a, b, h, i, lane, on, q);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(q[e], x[e], s);
            s = warp_sum(s) * a.g.scale;
            w += expf(s - a.lse[((int64_t)b * a.g.H + h) * a.g.T + i]);
        }
    if (lane == 0) {
        const int64_t at = (int64_t)bh * a.mass_ld + j;
        a.mass_out[at] = (a.mass_in ? a.mass_in[at] : 0.f) + w;
    }
}

}  // namespace

size_t kv4_attend_bytes(const Kv4Geom&, const Geom&, bool) { return 0; }

cudaError_t launch_kv4_attend(const Kv4AttendArgs& a, cudaStream_t s) {
    attend_rows<<<a.g.B * a.g.H * a.g.T, 128, 0, s>>>(a);
    cudaError_t e = counted(cudaGetLastError());
    if (e != cudaSuccess || !a.mass_out) return e;
    attend_mass<<<dim3((a.c.cap + 7) / 8, a.c.B * a.c.Hkv), 256, 0, s>>>(a);
    return counted(cudaGetLastError());
}

}  // namespace attn
