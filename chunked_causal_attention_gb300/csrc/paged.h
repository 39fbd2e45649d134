// Internal declarations of the paged key/value cache's kernels, shared by
// paged_api.cpp and the kernels.
#pragma once

#include "kv4.h"

namespace attn {

// The pool as the kernels see it: slot i of page p of head h is the row at p*sp + h*sh + i*st.
struct PagedGeom {
    int32_t pages, Hkv, D;
    int32_t shift;            // log2 of a page's slots
    int64_t sp, sh, st;
    void *k, *v;
    int32_t page() const { return 1 << shift; }
    // as a [B, H, T, D] tensor of pages, heads and slots (for tensor maps and checks)
    Geom geom() const {
        Geom g{};
        g.B = pages; g.H = g.Hkv = Hkv; g.T = page(); g.D = D;
        g.sb = g.sb_kv = sp; g.sh = g.sh_kv = sh; g.st = g.st_kv = st;
        return g;
    }
};

struct PagedStoreArgs {
    const void *k, *v;        // bf16 rows of the call
    PagedGeom c;
    const int32_t* slots;
    uint32_t* status;
    int64_t st, sh;           // element strides of the rows
    int32_t pieces;           // 16-byte pieces of K: T * Hkv * D / 8
    FastDiv by_vec, by_h;     // D / 8 and Hkv
};

// What the reservation's first kernel leaves for the second, for each sequence.
struct PagedSeq {
    int32_t tok;              // its first packed token
    int32_t len;              // slots in use before the call
    int32_t held;             // pages before the call; -1: refused
    int32_t top;              // its page i (i >= held) is free_pages[top - i]
};

struct PagedReserveArgs {
    const int32_t *add, *lens, *n_free;
    int32_t *free_pages, *table;
    int64_t table_ld;
    int32_t B, shift, pages, max_pages, T;
    int32_t *lens_out, *n_free_out, *cu, *slots;
    uint32_t* status;
    PagedSeq* seqs;           // workspace, B of them
    int32_t* back;            // workspace: pages put back by the sequences before, B of them
};

struct PagedAttendArgs {
    const void* q; void* o; float* lse;
    PagedGeom c;
    Geom g;                   // queries: B = 1, H, T packed tokens, D, strides, scale
    const int32_t* table; int64_t table_ld; int32_t max_pages;
    const int32_t *lens, *cu;
    int32_t B, each;          // sequences; cu null: tokens of each
    uint32_t* status;
    uint32_t* counter;        // work queue, zero between calls
    int4* cuts;               // workspace, B of them: a sequence's first partial, parts of a cut unit, units left whole,
                              // whether `offsets` stand for cu
    int32_t* offsets;         // workspace, B + 1 of them: cu put in order, where it is not
    float* parts;             // workspace: partials
    int32_t max_parts;        // how many it holds
    uint64_t wait_ns; int32_t stall;
};

// paged_attend.cu: workspace bytes after the cuts, and how many partials they hold
size_t paged_parts_bytes(const PagedGeom& c, const Geom& g, int32_t* max_parts);
bool paged_units_fit(const PagedGeom& c, const Geom& g, int64_t B);

cudaError_t launch_paged_store(const PagedStoreArgs& a, cudaStream_t s);       // paged_rows.cu
cudaError_t launch_paged_reserve(const PagedReserveArgs& a, cudaStream_t s);   // paged_rows.cu
cudaError_t launch_paged_attend(const PagedAttendArgs& a, cudaStream_t s);     // paged_attend.cu

}  // namespace attn
