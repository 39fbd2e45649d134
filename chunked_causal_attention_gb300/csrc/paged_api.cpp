// C-ABI layer of the paged key/value cache: argument validation, workspace layout
// and launches. No device memory is allocated here.
#include <algorithm>

#include "paged.h"

using namespace attn;

namespace {

constexpr size_t kAlign = 256;

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_ws(const void* ws, size_t have, size_t need) {
    if (!ws || have < need) return ATTN_E_WORKSPACE;
    return aligned(ws, kAlign) ? ATTN_OK : ATTN_E_ALIGN;
}

int launched(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_E_CUDA; }

// Most slots of a sequence: a tile more is still an int32.
constexpr int64_t kMaxSlots = INT32_MAX - 4096;

constexpr int64_t kMaxSeqs = 1 << 20;

// log2 of a page's slots, -1 if they are no power of two from 16 to 1024.
int page_shift(int64_t page) {
    for (int s = 4; s <= 10; ++s)
        if (page == 1ll << s) return s;
    return -1;
}

int check_cache(const attn_paged_cache* c, PagedGeom* g) {
    if (!c) return ATTN_E_INVAL;
    if (c->pages <= 0 || c->Hkv <= 0 || c->D <= 0 || page_shift(c->page) < 0) return ATTN_E_INVAL;
    if (c->pages > INT32_MAX / c->page || c->Hkv > (1 << 24)) return ATTN_E_INVAL;
    if (c->D < 8 || c->D > 256 || c->D % 8) return ATTN_E_UNSUPPORTED;
    if (c->sp <= 0 || c->sh <= 0 || c->st <= 0) return ATTN_E_INVAL;
    if (c->sp % 8 || c->sh % 8 || c->st % 8) return ATTN_E_ALIGN;
    if (!c->k || !c->v) return ATTN_E_INVAL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return ATTN_E_ALIGN;
    g->pages = (int32_t)c->pages; g->Hkv = (int32_t)c->Hkv; g->D = (int32_t)c->D;
    g->shift = page_shift(c->page);
    g->sp = c->sp; g->sh = c->sh; g->st = c->st;
    g->k = c->k; g->v = c->v;
    return rows_apart(g->geom()) ? ATTN_OK : ATTN_E_INVAL;
}

// Bytes between the first and the last element of rows with a shape's query strides.
size_t span(const Geom& g) {
    return 2 * ((size_t)(g.B - 1) * g.sb + (size_t)(g.H - 1) * g.sh + (size_t)(g.T - 1) * g.st + g.D);
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

// Queries (attend) or rows (store) of packed tokens over this cache.
int packed_geom(const attn_shape* shape, const PagedGeom& c, Geom* g) {
    int st = shape_geom(shape, g);
    if (st) return st;
    return g->B == 1 && g->D == c.D ? ATTN_OK : ATTN_E_INVAL;
}

int attend_geom(const attn_shape* shape, const PagedGeom& c, int64_t B, Geom* g) {
    int st = packed_geom(shape, c, g);
    if (st) return st;
    if (B <= 0 || B > kMaxSeqs || g->H % c.Hkv || !rows_apart(*g)) return ATTN_E_INVAL;
    g->Hkv = c.Hkv;
    return (int64_t)g->H * g->T <= INT32_MAX && paged_units_fit(c, *g, B) ? ATTN_OK : ATTN_E_INVAL;
}

// What the tile kernel of attention notes of its sequences: cuts, and offsets put in order.
size_t cuts_bytes(int64_t B) { return round_up((size_t)B * sizeof(int4), kAlign); }
size_t notes_bytes(int64_t B) { return cuts_bytes(B) + round_up((size_t)(B + 1) * sizeof(int32_t), kAlign); }

size_t seqs_bytes(int64_t B) { return round_up((size_t)B * sizeof(PagedSeq), kAlign); }

size_t reserve_bytes(int64_t B) { return kHeaderBytes + seqs_bytes(B) + round_up((size_t)B * sizeof(int32_t), kAlign); }

}  // namespace

extern "C" {

int attn_paged_workspace_size(const attn_paged_cache* cache, const attn_shape* shape, int64_t B, int32_t op,
                              size_t* bytes) {
    if (!bytes) return ATTN_E_INVAL;
    if (op == ATTN_PAGED_RESERVE) {
        if (B <= 0 || B > kMaxSeqs) return ATTN_E_INVAL;
        *bytes = reserve_bytes(B);
        return ATTN_OK;
    }
    PagedGeom c;
    int st = check_cache(cache, &c);
    if (st) return st;
    if (op == ATTN_PAGED_STORE) {
        *bytes = kHeaderBytes;
    } else if (op == ATTN_PAGED_ATTEND) {
        Geom g;
        if ((st = attend_geom(shape, c, B, &g))) return st;
        int32_t n;
        *bytes = kHeaderBytes + notes_bytes(B) + round_up(paged_parts_bytes(c, g, &n), kAlign);
    } else {
        return ATTN_E_INVAL;
    }
    return ATTN_OK;
}

int attn_paged_reserve(const int32_t* add, const int32_t* lens, int64_t B, int64_t page, int64_t pages,
                       const int32_t* n_free, int32_t* free_pages, int32_t* table, int64_t table_ld,
                       int64_t max_pages, int32_t* lens_out, int32_t* n_free_out, int32_t* cu_seqlens,
                       int32_t* slots, int64_t T, void* ws, size_t ws_bytes, void* stream) {
    PagedReserveArgs a;
    a.shift = page_shift(page);
    if (a.shift < 0 || B <= 0 || B > kMaxSeqs || T <= 0 || T > INT32_MAX / 2) return ATTN_E_INVAL;
    if (pages <= 0 || pages > INT32_MAX / page || max_pages <= 0 || max_pages > kMaxSlots / page) return ATTN_E_INVAL;
    if (table_ld < max_pages || table_ld > INT64_MAX / 8 / B) return ATTN_E_INVAL;
    const void* p[] = {add, lens, n_free, free_pages, table, lens_out, n_free_out, cu_seqlens, slots};
    for (const void* x : p)
        if (!x) return ATTN_E_INVAL;
    for (const void* x : p)
        if (!aligned(x, 4)) return ATTN_E_ALIGN;
    // what is written lies apart from all the rest; lens_out may be lens and n_free_out n_free
    struct Range { const void* p; size_t n; bool out; };
    const size_t w = sizeof(int32_t), nt = ((size_t)(B - 1) * table_ld + max_pages) * w;
    enum { ADD, LENS, N_FREE, FREE, TABLE, LENS_OUT, N_FREE_OUT, CU, SLOTS, RANGES };
    const Range r[RANGES] = {{add, B * w, false}, {lens, B * w, false}, {n_free, w, false}, {free_pages, pages * w, true},
                             {table, nt, true}, {lens_out, B * w, true}, {n_free_out, w, true},
                             {cu_seqlens, (B + 1) * w, true}, {slots, T * w, true}};
    for (int i = 0; i < RANGES; ++i)
        for (int j = 0; j < i; ++j) {
            const bool in_place = r[i].p == r[j].p && ((i == LENS_OUT && j == LENS) || (i == N_FREE_OUT && j == N_FREE));
            if ((r[i].out || r[j].out) && !in_place && overlap(r[i].p, r[i].n, r[j].p, r[j].n)) return ATTN_E_INVAL;
        }
    int st = check_ws(ws, ws_bytes, reserve_bytes(B));
    if (st) return st;
    a.add = add; a.lens = lens; a.n_free = n_free;
    a.free_pages = free_pages; a.table = table; a.table_ld = table_ld;
    a.B = (int32_t)B; a.pages = (int32_t)pages; a.max_pages = (int32_t)max_pages; a.T = (int32_t)T;
    a.lens_out = lens_out; a.n_free_out = n_free_out; a.cu = cu_seqlens; a.slots = slots;
    a.status = (uint32_t*)ws;
    a.seqs = (PagedSeq*)((uint8_t*)ws + kHeaderBytes);
    a.back = (int32_t*)((uint8_t*)ws + kHeaderBytes + seqs_bytes(B));
    return launched(launch_paged_reserve(a, (cudaStream_t)stream));
}

int attn_paged_store(const void* k, const void* v, const attn_shape* shape, const attn_paged_cache* cache,
                     const int32_t* slots, void* ws, size_t ws_bytes, void* stream) {
    PagedStoreArgs a;
    Geom g;
    int st = check_cache(cache, &a.c);
    if (st) return st;
    if ((st = packed_geom(shape, a.c, &g))) return st;
    if (!k || !v || !slots || g.H != a.c.Hkv) return ATTN_E_INVAL;
    const int64_t rows = (int64_t)g.H * g.T;
    if (rows > INT32_MAX || rows * (g.D / 8) > INT32_MAX) return ATTN_E_INVAL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return ATTN_E_ALIGN;
    if ((st = check_ws(ws, ws_bytes, kHeaderBytes))) return st;
    a.k = k; a.v = v;
    a.slots = slots;
    a.status = (uint32_t*)ws;
    a.st = g.st; a.sh = g.sh;
    a.pieces = (int32_t)(rows * (g.D / 8));
    a.by_vec = FastDiv::of((uint32_t)g.D / 8);
    a.by_h = FastDiv::of((uint32_t)g.H);
    return launched(launch_paged_store(a, (cudaStream_t)stream));
}

int attn_paged_attend(const void* q, const attn_shape* shape, const attn_paged_cache* cache, const int32_t* table,
                      int64_t table_ld, int64_t max_pages, const int32_t* lens, const int32_t* cu_seqlens, int64_t B,
                      void* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
    PagedAttendArgs a;
    int st = check_cache(cache, &a.c);
    if (st) return st;
    if ((st = attend_geom(shape, a.c, B, &a.g))) return st;
    if (!q || !table || !lens || !o || !lse) return ATTN_E_INVAL;
    if (max_pages <= 0 || max_pages > (kMaxSlots >> a.c.shift) || table_ld < max_pages || table_ld > INT64_MAX / 8 / B)
        return ATTN_E_INVAL;
    if (!cu_seqlens && a.g.T % B) return ATTN_E_INVAL;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
        !aligned(cu_seqlens, 4))
        return ATTN_E_ALIGN;
    if (overlap(q, span(a.g), o, span(a.g))) return ATTN_E_INVAL;
    size_t parts = paged_parts_bytes(a.c, a.g, &a.max_parts);
    if ((st = check_ws(ws, ws_bytes, kHeaderBytes + notes_bytes(B) + round_up(parts, kAlign)))) return st;
    a.q = q; a.o = o; a.lse = lse;
    a.table = table; a.table_ld = table_ld; a.max_pages = (int32_t)max_pages;
    a.lens = lens; a.cu = cu_seqlens;
    a.B = (int32_t)B; a.each = (int32_t)(a.g.T / B);
    a.status = &((WsHeader*)ws)->status;
    a.counter = &((WsHeader*)ws)->counter[2];
    a.cuts = (int4*)((uint8_t*)ws + kHeaderBytes);
    a.offsets = (int32_t*)((uint8_t*)ws + kHeaderBytes + cuts_bytes(B));
    a.parts = (float*)((uint8_t*)ws + kHeaderBytes + notes_bytes(B));
    wait_settings(&a.wait_ns, &a.stall);
    return launched(launch_paged_attend(a, (cudaStream_t)stream));
}

}  // extern "C"
