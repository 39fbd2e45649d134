// Internal declarations of the 4-bit key/value cache's kernels and of the key
// mass, shared by kv4_api.cpp and the kernels.
#pragma once

#include "attn_internal.h"

namespace attn {

constexpr int kKv4Block = 16;   // dims per e4m3 scale

// The cache as the kernels see it: row r = b*sb + h*sh + t, codes at r*cb, scales at r*nb.
struct Kv4Geom {
    int32_t B, Hkv, cap, D;
    int64_t sb, sh;
    uint8_t *kc, *ks, *vc, *vs;
    float k_scale, v_scale;
    int32_t cb;   // bytes of a row's codes, D / 2
    int32_t nb;   // bytes of a row's scales, ceil(D / 16)
};

// n / d for 0 <= n < 2^31 by a multiplication: with p = 31 + ceil(log2 d) and
// m = ceil(2^p / d) < 2^32, floor(n m / 2^p) = floor(n / d) (Granlund and Montgomery).
struct FastDiv {
    uint32_t d, m, s;
    static FastDiv of(uint32_t d) {
        uint32_t l = 0;
        while ((1ull << l) < d) ++l;
        const uint32_t p = 31 + l;
        return FastDiv{d, (uint32_t)(((1ull << p) + d - 1) / d), p - 32};
    }
#ifdef __CUDACC__
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return d == 1 ? n : __umulhi(n, m) >> s; }
#endif
};

struct Kv4RowsArgs {
    void *k, *v;              // bf16 rows, read by the store and written by the load
    Kv4Geom c;
    const int32_t* pos;
    const int32_t* cu;        // null: dense
    uint32_t* status;
    int64_t sb, st, sh;       // element strides of k, v
    int64_t rows;             // rows in all: B * Hkv * T dense, T * Hkv packed
    FastDiv by_t, by_h;       // T (dense) and Hkv
};

struct Kv4AttendArgs {
    const void* q; void* o; float* lse;
    Kv4Geom c;
    Geom g;                   // queries: B, H, T = new tokens, D, strides, scale
    const int32_t* lens;
    const float* mass_in; float* mass_out; int64_t mass_ld;
    uint32_t* status;
    float* parts;             // workspace after the header
    int32_t grid;             // CTAs of the split kernel, the workspace was sized for
};

struct Kv4EvictArgs {
    Kv4Geom src, dst;
    const int32_t* lens; int32_t* lens_out;
    const float* mass; int64_t mass_ld;
    float* mass_out; int64_t mass_out_ld;
    int32_t keep, recent;
    int32_t* slots;
    uint32_t* status;
};

// Keys [j0, j1) of a key/value head, at most 128; the chunks whose rows may see them
// are among [c_lo, c_hi).
struct MassItem {
    int32_t j0, j1, c_lo, c_hi;
};

struct MassArgs {
    const void* q; const void* k; const float* lse;
    const float* mass_in; float* mass_out;
    const attn_chunk* chunks; int32_t n;   // in the workspace
    const MassItem* items; int32_t n_items;
    uint32_t* status;
    uint32_t* counter;
    uint64_t wait_ns; int32_t stall;
    Geom g;
};

// Workspace bytes of attn_key_mass on these (valid) chunks, kv4_api.cpp.
size_t key_mass_bytes(const Geom& g, const attn_chunk* c, int32_t n);

// kv4_attend.cu: bytes after the header
size_t kv4_attend_bytes(const Kv4Geom& c, const Geom& g, bool mass);

cudaError_t launch_kv4_store(const Kv4RowsArgs& a, cudaStream_t s);    // kv4_rows.cu
cudaError_t launch_kv4_load(const Kv4RowsArgs& a, cudaStream_t s);     // kv4_rows.cu
cudaError_t launch_kv4_attend(const Kv4AttendArgs& a, cudaStream_t s); // kv4_attend.cu
cudaError_t launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t s);   // kv4_evict.cu
cudaError_t launch_key_mass(const MassArgs& a, cudaStream_t s);        // key_mass.cu
// One chunk of few rows over many keys: whether these chunks (host) are that, and its kernel.
bool key_mass_window(const MassArgs& a, const attn_chunk* chunks);
cudaError_t launch_key_mass_window(const MassArgs& a, const attn_chunk& ch, cudaStream_t s);

// attn_api.cpp's argument rules, for the entry points in kv4_api.cpp
int shape_geom(const attn_shape* s, Geom* g);
// kv4_api.cpp: whether rows with these strides, of D elements each, lie apart: a call
// that writes them may have no two in the same memory.
bool rows_apart(const Geom& g);
int chunks_fwd_status(const attn_chunk* c, int32_t n, int32_t T);

}  // namespace attn
