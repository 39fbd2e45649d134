// C-ABI layer of the 4-bit key/value cache and of the key mass: argument
// validation, workspace layout and launches. No device memory is allocated here.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <numeric>
#include <vector>

#include "kv4.h"

using namespace attn;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxLd = 1ll << 36;   // floats between two rows of weights; with 2^24 rows offsets stay below 2^63

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_ws(const void* ws, size_t have, size_t need) {
    if (!ws || have < need) return ATTN_E_WORKSPACE;
    return aligned(ws, kAlign) ? ATTN_OK : ATTN_E_ALIGN;
}

int launched(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_E_CUDA; }

// A power of two in [2^-64, 2^64].
bool tensor_scale_ok(float x) {
    int e = 0;
    return std::isfinite(x) && x > 0.f && std::frexp(x, &e) == 0.5f && e >= -63 && e <= 65;
}

int check_cache(const attn_kv4_cache* c, Kv4Geom* g) {
    if (!c) return ATTN_E_INVAL;
    if (c->B <= 0 || c->Hkv <= 0 || c->cap <= 0 || c->D <= 0) return ATTN_E_INVAL;
    if (c->B > INT32_MAX || c->Hkv > INT32_MAX || c->cap > INT32_MAX - 1024 || c->B * c->Hkv > (1ll << 24))
        return ATTN_E_INVAL;
    if (c->D < 8 || c->D > 256 || c->D % 8) return ATTN_E_UNSUPPORTED;
    if (!tensor_scale_ok(c->k_scale) || !tensor_scale_ok(c->v_scale)) return ATTN_E_INVAL;
    if (c->sb <= 0 || c->sh <= 0) return ATTN_E_INVAL;
    // rows of different sequences and heads are different rows: the heads of a sequence lie between two sequences,
    // or the sequences of a head between two heads
    if (c->sb > INT64_MAX / c->B / 4 || c->sh > INT64_MAX / c->Hkv / 4) return ATTN_E_INVAL;
    if (c->sh < c->cap && c->Hkv > 1) return ATTN_E_INVAL;
    if (c->sb < c->cap && c->B > 1) return ATTN_E_INVAL;
    if (c->B > 1 && c->Hkv > 1 && c->sb < (c->Hkv - 1) * c->sh + c->cap && c->sh < (c->B - 1) * c->sb + c->cap)
        return ATTN_E_INVAL;
    if (c->cap % 16 || c->sb % 16 || c->sh % 16) return ATTN_E_ALIGN;
    const void* p[] = {c->k_codes, c->k_scales, c->v_codes, c->v_scales};
    for (const void* x : p)
        if (!x) return ATTN_E_INVAL;
    for (const void* x : p)
        if (!aligned(x, 16)) return ATTN_E_ALIGN;
    g->B = (int32_t)c->B; g->Hkv = (int32_t)c->Hkv; g->cap = (int32_t)c->cap; g->D = (int32_t)c->D;
    g->sb = c->sb; g->sh = c->sh;
    g->kc = (uint8_t*)c->k_codes; g->ks = (uint8_t*)c->k_scales;
    g->vc = (uint8_t*)c->v_codes; g->vs = (uint8_t*)c->v_scales;
    g->k_scale = c->k_scale; g->v_scale = c->v_scale;
    g->cb = g->D / 2;
    g->nb = (g->D + kKv4Block - 1) / kKv4Block;
    return ATTN_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

// Rows from the first to the last of a cache, gaps between them included.
size_t span_rows(const Kv4Geom& c) {
    return (size_t)(c.B - 1) * c.sb + (size_t)(c.Hkv - 1) * c.sh + c.cap;
}

// Whether stretches of na bytes at a and of nb bytes at b, each repeated at multiples of `period` bytes, never
// meet: slots of one allocation taken as two caches lie between one another without overlapping.
bool apart(const void* a, size_t na, const void* b, size_t nb, size_t period) {
    if (!period) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    const size_t d = y >= x ? (y - x) % period : (period - (x - y) % period) % period;
    return d >= na && d + nb <= period;
}

bool overlap(const Kv4Geom& a, const Kv4Geom& b) {
    const size_t ra = span_rows(a), rb = span_rows(b);
    // rows that divide the distances between all heads and sequences
    int64_t g = 0;
    for (const Kv4Geom* c : {&a, &b}) {
        if (c->B > 1) g = std::gcd(g, c->sb);
        if (c->Hkv > 1) g = std::gcd(g, c->sh);
    }
    struct Arr { const void* p; int32_t row; };
    const Arr x[] = {{a.kc, a.cb}, {a.ks, a.nb}, {a.vc, a.cb}, {a.vs, a.nb}};
    const Arr y[] = {{b.kc, b.cb}, {b.ks, b.nb}, {b.vc, b.cb}, {b.vs, b.nb}};
    for (const Arr& p : x)
        for (const Arr& q : y)
            if (overlap(p.p, ra * p.row, q.p, rb * q.row) &&
                !(p.row == q.row && apart(p.p, (size_t)a.cap * p.row, q.p, (size_t)b.cap * q.row, (size_t)g * p.row)))
                return true;
    return false;
}

// Rows of weights, a of na floats `lda` apart and b of nb floats `ldb` apart.
bool mass_overlap(const float* a, int64_t na, int64_t lda, const float* b, int64_t nb, int64_t ldb, int64_t rows) {
    return overlap(a, ((rows - 1) * lda + na) * 4, b, ((rows - 1) * ldb + nb) * 4) &&
           !(rows > 1 && apart(a, na * 4, b, nb * 4, (size_t)std::gcd(lda, ldb) * 4));
}

// mass_in null, equal to mass_out, or apart from it.
int check_mass(const float* in, const float* out, int64_t floats, int64_t ld, int64_t rows) {
    if (!aligned(in, 16) || !aligned(out, 16)) return ATTN_E_ALIGN;
    if (in && in != out && mass_overlap(in, floats, ld, out, floats, ld, rows)) return ATTN_E_INVAL;
    return ATTN_OK;
}

// Whether rows with these strides, of D elements each, lie apart: a call writes them, so no two may share memory.
bool rows_apart(const Geom& g) {
    struct Dim { int64_t stride, n; };
    Dim d[] = {{g.sb, g.B}, {g.sh, g.H}, {g.st, g.T}};
    std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    __int128 extent = g.D;
    for (const Dim& x : d) {
        if (x.n == 1) continue;
        if (x.stride < extent) return false;
        extent += (__int128)x.stride * (x.n - 1);
    }
    return true;
}

int rows_common(const void* k, const void* v, const attn_shape* shape, const attn_kv4_cache* cache,
                const int32_t* pos, const int32_t* cu, void* ws, size_t ws_bytes, cudaStream_t s, bool store) {
    Kv4RowsArgs a;
    Geom g;
    int st = check_cache(cache, &a.c);
    if (st) return st;
    if ((st = shape_geom(shape, &g))) return st;
    if (!k || !v || !pos) return ATTN_E_INVAL;
    if (g.D != a.c.D || g.H != a.c.Hkv || g.B != (cu ? 1 : a.c.B)) return ATTN_E_INVAL;
    if (!store && !rows_apart(g)) return ATTN_E_INVAL;
    a.rows = (int64_t)g.B * g.H * g.T;
    if (a.rows > INT32_MAX) return ATTN_E_INVAL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(pos, 4) || !aligned(cu, 4)) return ATTN_E_ALIGN;
    if ((st = check_ws(ws, ws_bytes, kHeaderBytes))) return st;
    a.k = const_cast<void*>(k); a.v = const_cast<void*>(v);
    a.pos = pos; a.cu = cu;
    a.status = (uint32_t*)ws;
    a.sb = g.sb; a.st = g.st; a.sh = g.sh;
    a.by_t = FastDiv::of((uint32_t)g.T);
    a.by_h = FastDiv::of((uint32_t)g.H);
    return launched(store ? launch_kv4_store(a, s) : launch_kv4_load(a, s));
}

int attend_geom(const attn_shape* shape, const Kv4Geom& c, Geom* g) {
    int st = shape_geom(shape, g);
    if (st) return st;
    if (g->D != c.D || g->B != c.B || g->H % c.Hkv) return ATTN_E_INVAL;
    if (!rows_apart(*g)) return ATTN_E_INVAL;
    // the queries' rows are numbered in 31 bits
    if ((int64_t)g->B * g->H * g->T > INT32_MAX) return ATTN_E_INVAL;
    g->Hkv = c.Hkv;
    return ATTN_OK;
}

}  // namespace

// Key tiles of attn_key_mass, those that the most rows see first. Chunks are sorted
// by rows, so the ones that end after a tile's first key are a tail of the table; of
// those, the last that starts its context before the tile's end bounds the range.
static std::vector<MassItem> mass_items(const Geom& g, const attn_chunk* c, int32_t n) {
    std::vector<int32_t> least(n + 1, INT32_MAX);       // least context start of the chunks [i, n)
    std::vector<int64_t> rows(n + 1, 0);                // rows of the chunks [0, i)
    for (int32_t i = n - 1; i >= 0; --i) least[i] = std::min(least[i + 1], c[i].ctx_begin);
    for (int32_t i = 0; i < n; ++i) rows[i + 1] = rows[i] + (c[i].q_end - c[i].q_begin);
    struct Costed { MassItem it; int64_t cost; };
    std::vector<Costed> v;
    int32_t lo = 0, hi = 0;
    for (int32_t j0 = 0; j0 < g.T; j0 += std::min(kTile, g.T - j0)) {
        const int32_t j1 = j0 + std::min(kTile, g.T - j0);
        while (lo < n && c[lo].q_end <= j0) ++lo;
        while (hi < n && least[hi] < j1) ++hi;
        Costed x{{j0, j1, lo, std::max(lo, hi)}, 0};
        if (lo < hi) x.cost = rows[hi] - rows[lo] - std::max(0, j0 - c[lo].q_begin);
        v.push_back(x);
    }
    std::stable_sort(v.begin(), v.end(), [](const Costed& a, const Costed& b) { return a.cost > b.cost; });
    std::vector<MassItem> items(v.size());
    for (size_t i = 0; i < v.size(); ++i) items[i] = v[i].it;
    return items;
}

static size_t mass_items_offset(int32_t n) { return kHeaderBytes + round_up((size_t)n * sizeof(attn_chunk), kAlign); }

size_t attn::key_mass_bytes(const Geom& g, const attn_chunk*, int32_t n) {
    return mass_items_offset(n) + round_up(((size_t)g.T + kTile - 1) / kTile * sizeof(MassItem), kAlign);
}

extern "C" {

int attn_kv4_workspace_size(const attn_kv4_cache* cache, const attn_shape* shape, int32_t op, size_t* bytes) {
    Kv4Geom c;
    if (!bytes) return ATTN_E_INVAL;
    int st = check_cache(cache, &c);
    if (st) return st;
    if (op == ATTN_KV4_ROWS) {
        *bytes = kHeaderBytes;
    } else if (op == ATTN_KV4_ATTEND || op == ATTN_KV4_ATTEND_MASS) {
        Geom g;
        if ((st = attend_geom(shape, c, &g))) return st;
        *bytes = kHeaderBytes + round_up(kv4_attend_bytes(c, g, op == ATTN_KV4_ATTEND_MASS), kAlign);
    } else {
        return ATTN_E_INVAL;
    }
    return ATTN_OK;
}

int attn_kv4_store(const void* k, const void* v, const attn_shape* shape, const attn_kv4_cache* cache,
                   const int32_t* pos, const int32_t* cu_seqlens, void* ws, size_t ws_bytes, void* stream) {
    return rows_common(k, v, shape, cache, pos, cu_seqlens, ws, ws_bytes, (cudaStream_t)stream, true);
}

int attn_kv4_load(const attn_kv4_cache* cache, const int32_t* pos, const int32_t* cu_seqlens,
                  const attn_shape* shape, void* k, void* v, void* ws, size_t ws_bytes, void* stream) {
    return rows_common(k, v, shape, cache, pos, cu_seqlens, ws, ws_bytes, (cudaStream_t)stream, false);
}

int attn_kv4_attend(const void* q, const attn_shape* shape, const attn_kv4_cache* cache, const int32_t* lens,
                    void* o, float* lse, const float* mass_in, float* mass_out, int64_t mass_ld,
                    void* ws, size_t ws_bytes, void* stream) {
    Kv4AttendArgs a;
    int st = check_cache(cache, &a.c);
    if (st) return st;
    if ((st = attend_geom(shape, a.c, &a.g))) return st;
    if (!q || !lens || !o || !lse) return ATTN_E_INVAL;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 16) || !aligned(lens, 4)) return ATTN_E_ALIGN;
    if (mass_out) {
        if (mass_ld <= 0 || mass_ld > kMaxLd) return ATTN_E_INVAL;
        if ((st = check_mass(mass_in, mass_out, std::min<int64_t>(mass_ld, a.c.cap), mass_ld, (int64_t)a.c.B * a.c.Hkv)))
            return st;
    } else if (mass_in) {
        return ATTN_E_INVAL;
    }
    if ((st = check_ws(ws, ws_bytes, kHeaderBytes + round_up(kv4_attend_bytes(a.c, a.g, mass_out != nullptr), kAlign))))
        return st;
    a.q = q; a.o = o; a.lse = lse; a.lens = lens;
    a.mass_in = mass_in; a.mass_out = mass_out; a.mass_ld = mass_ld;
    a.status = (uint32_t*)ws;
    a.parts = (float*)((uint8_t*)ws + kHeaderBytes);
    return launched(launch_kv4_attend(a, (cudaStream_t)stream));
}

int attn_kv4_evict(const attn_kv4_cache* src, const int32_t* lens, const float* mass, int64_t mass_ld,
                   int32_t keep, int32_t recent, const attn_kv4_cache* dst, int32_t* lens_out,
                   float* mass_out, int64_t mass_out_ld, int32_t* slots,
                   void* ws, size_t ws_bytes, void* stream) {
    Kv4EvictArgs a;
    int st = check_cache(src, &a.src);
    if (st) return st;
    if ((st = check_cache(dst, &a.dst))) return st;
    if (!lens || !mass || !lens_out || !slots) return ATTN_E_INVAL;
    if (a.src.B != a.dst.B || a.src.Hkv != a.dst.Hkv || a.src.D != a.dst.D || a.src.k_scale != a.dst.k_scale ||
        a.src.v_scale != a.dst.v_scale)
        return ATTN_E_INVAL;
    if (keep < 1 || keep > a.dst.cap || recent < 0 || mass_ld <= 0 || mass_ld > kMaxLd ||
        (mass_out && (mass_out_ld < keep || mass_out_ld > kMaxLd)))
        return ATTN_E_INVAL;
    if (!aligned(mass, 16) || !aligned(mass_out, 16) || !aligned(slots, 4) || !aligned(lens, 4) || !aligned(lens_out, 4))
        return ATTN_E_ALIGN;
    if ((int64_t)a.src.B * a.src.Hkv * keep > INT32_MAX) return ATTN_E_INVAL;
    if (overlap(a.src, a.dst)) return ATTN_E_INVAL;
    if (mass_out && mass_overlap(mass, std::min<int64_t>(mass_ld, a.src.cap), mass_ld, mass_out, keep, mass_out_ld,
                                 (int64_t)a.src.B * a.src.Hkv))
        return ATTN_E_INVAL;
    if ((st = check_ws(ws, ws_bytes, kHeaderBytes))) return st;
    a.lens = lens; a.lens_out = lens_out;
    a.mass = mass; a.mass_ld = mass_ld;
    a.mass_out = mass_out; a.mass_out_ld = mass_out_ld;
    a.keep = keep; a.recent = recent;
    a.slots = slots;
    a.status = (uint32_t*)ws;
    return launched(launch_kv4_evict(a, (cudaStream_t)stream));
}

int attn_key_mass(const void* q, const void* k, const float* lse, const attn_chunk* chunks, int32_t n,
                  const attn_shape* shape, const float* mass_in, float* mass_out,
                  void* ws, size_t ws_bytes, void* stream) {
    MassArgs a;
    int st = shape_geom(shape, &a.g);
    if (st) return st;
    if ((st = chunks_fwd_status(chunks, n, a.g.T))) return st;
    if (!q || !k || !lse || !mass_out) return ATTN_E_INVAL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(lse, 16)) return ATTN_E_ALIGN;
    if ((st = check_mass(mass_in, mass_out, (int64_t)a.g.B * a.g.Hkv * a.g.T, 0, 1))) return st;
    if ((st = check_ws(ws, ws_bytes, key_mass_bytes(a.g, chunks, n)))) return st;
    cudaStream_t s = (cudaStream_t)stream;
    uint8_t* w = (uint8_t*)ws;
    a.q = q; a.k = k; a.lse = lse; a.mass_in = mass_in; a.mass_out = mass_out;
    a.chunks = (const attn_chunk*)(w + kHeaderBytes);
    a.n = n;
    a.items = (const MassItem*)(w + mass_items_offset(n));
    a.n_items = 0;
    a.status = (uint32_t*)ws;
    a.counter = &((WsHeader*)ws)->counter[0];
    wait_settings(&a.wait_ns, &a.stall);
    if (key_mass_window(a, chunks)) {
        if (cudaMemsetAsync(ws, 0, kHeaderBytes, s) != cudaSuccess) return ATTN_E_CUDA;
        return launched(launch_key_mass_window(a, chunks[0], s));
    }
    try {
        // the zeroed header, the chunks and the items in one copy
        const std::vector<MassItem> items = mass_items(a.g, chunks, n);
        const size_t off = mass_items_offset(n), bytes = off + items.size() * sizeof(MassItem);
        std::vector<uint8_t> lists(bytes, 0);
        if (n) std::memcpy(lists.data() + kHeaderBytes, chunks, (size_t)n * sizeof(attn_chunk));
        std::memcpy(lists.data() + off, items.data(), items.size() * sizeof(MassItem));
        if (launch_upload(w, lists.data(), bytes, s) != cudaSuccess) return ATTN_E_CUDA;
        a.n_items = (int32_t)items.size();
    } catch (const std::bad_alloc&) {
        return ATTN_E_CUDA;
    }
    return launched(launch_key_mass(a, s));
}

}  // extern "C"
