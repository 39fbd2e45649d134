// The attention weight of each key over query rows: the simple form, one warp per key.
#include "kv4_device.cuh"

namespace attn {
namespace {

__global__ void __launch_bounds__(256) key_mass_rows(const MassArgs a) {
    const int lane = threadIdx.x & 31;
    const int j = blockIdx.x * 8 + (threadIdx.x >> 5), bh = blockIdx.y;
    const int b = bh / a.g.Hkv, hk = bh % a.g.Hkv, G = a.g.H / a.g.Hkv;
    if (j >= a.g.T) return;
    const bool on = lane * 8 < a.g.D;
    float x[8], w = 0.f;
    const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(a.k) + (int64_t)b * a.g.sb_kv +
                             (int64_t)hk * a.g.sh_kv + (int64_t)j * a.g.st_kv;
    for (int e = 0; e < 8; ++e) x[e] = on ? __bfloat162float(k[lane * 8 + e]) : 0.f;
    for (int c = 0; c < a.n; ++c) {
        const attn_chunk ch = a.chunks[c];
        if (j < ch.ctx_begin || j >= ch.q_end) continue;
        for (int h = hk * G; h < hk * G + G; ++h)
            for (int t = max(ch.q_begin, j); t < ch.q_end; ++t) {
                const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + (int64_t)b * a.g.sb +
                                         (int64_t)h * a.g.sh + (int64_t)t * a.g.st;
                float s = 0.f;
                if (on)
                    for (int e = 0; e < 8; ++e) s = fmaf(__bfloat162float(q[lane * 8 + e]), x[e], s);
                for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                const float lse = a.lse[((int64_t)b * a.g.H + h) * a.g.T + t];
                w += lse == -INFINITY ? 0.f : expf(s * a.g.scale - lse);
            }
    }
    if (lane == 0) {
        const int64_t at = (int64_t)bh * a.g.T + j;
        a.mass_out[at] = (a.mass_in ? a.mass_in[at] : 0.f) + w;
    }
}

}  // namespace

cudaError_t launch_key_mass(const MassArgs& a, cudaStream_t s) {
    key_mass_rows<<<dim3((a.g.T + 7) / 8, a.g.B * a.g.Hkv), 256, 0, s>>>(a);
    return counted(cudaGetLastError());
}

}  // namespace attn
