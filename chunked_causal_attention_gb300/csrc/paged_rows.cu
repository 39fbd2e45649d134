// The paged cache's bookkeeping and its rows: reserve slots for the next tokens,
// store rows in them.
//
// Reserve. Three prefix sums over the sequences (pages put back, pages taken, tokens)
// by one block, which also writes the lengths, the offsets and the stack's height and
// puts the pages of ended sequences back; then one thread a token finds its sequence
// by bisection of the offsets and its slot from the table, or from the stack for a new
// page, whose first token writes it into the table. A decode step's few tokens are
// taken by the block itself, so that the call is one launch: it is bound by latency
// (reads of add and lens, three block-wide steps, reads of table or stack). Measured: one
// token for each of 64 sequences 3.8 us, 40007 tokens of 512 sequences 8.8 us, 131072
// tokens of 8 sequences 5.1 us.
//
// Store. A copy: a thread moves 16-byte pieces of keys and values, four of each in
// flight; bound by memory. Measured: 16384 rows of 32 heads of 128 dims 80.7 us (6.65
// TB/s, 98% of the copy rate), 64 rows of 8 heads 2.6 us.
#include <algorithm>

#include "kv4_device.cuh"
#include "paged.h"

namespace attn {
namespace {

using kv4::grid_go;
using kv4::grid_wait;
using kv4::launch_early;

// ------------------------------------------------------------------ reserve

constexpr int kPlanThreads = 1024;
constexpr int kPlanSeqs = 1024;          // sequences whose records the first kernel keeps in shared memory
// Calls of at most so many tokens are one launch: 64 sequences' 4096 tokens 6.0 us and 5.5 by two, 1024 3.8 and 5.5,
// 8192 8.8 and 5.7; a second launch is 2 us of the host's time.
constexpr int kInlineTokens = 4096;
constexpr int kSlotThreads = 256;

// Slot of packed token t, -1 if it has none. cu: where the sequences begin, ascending.
__device__ __forceinline__ int32_t slot_of(const PagedReserveArgs& a, const PagedSeq* seqs, int32_t total, int32_t t) {
    if (t >= total) return -1;
    int32_t lo = 0, hi = a.B;                        // the last sequence that begins at or before t
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (seqs[mid].tok <= t) lo = mid; else hi = mid;
    }
    const PagedSeq q = seqs[lo];
    if (q.held < 0) return -1;
    const int32_t s = q.len + (t - q.tok), i = s >> a.shift;
    int32_t* entry = a.table + (int64_t)lo * a.table_ld + i;
    int32_t id;
    if (i < q.held) {
        id = *entry;
    } else {
        id = a.free_pages[q.top - i];
        if ((s & ((1 << a.shift) - 1)) == 0) *entry = id;          // a new page's first slot is a new token's
    }
    if ((uint32_t)id >= (uint32_t)a.pages) {
        set_error(a.status, ATTN_E_BOUNDS);
        return -1;
    }
    return (id << a.shift) | (s & ((1 << a.shift) - 1));
}

// Sums of three numbers over the threads before this one, and over all.
struct Three {
    int64_t back, need, tok;
};

// Inclusive over the lanes of a warp.
__device__ __forceinline__ Three warp_scan3(Three y) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t p = __shfl_up_sync(0xffffffffu, y.back, m), q = __shfl_up_sync(0xffffffffu, y.need, m),
                      r = __shfl_up_sync(0xffffffffu, y.tok, m);
        if (lane >= m) {
            y.back += p;
            y.need += q;
            y.tok += r;
        }
    }
    return y;
}

__device__ __forceinline__ Three lane_of(const Three& x, int lane) {
    return Three{__shfl_sync(0xffffffffu, x.back, lane), __shfl_sync(0xffffffffu, x.need, lane),
                 __shfl_sync(0xffffffffu, x.tok, lane)};
}

__device__ __forceinline__ Three scan3(const Three& x, Three& all, Three* scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Three y = warp_scan3(x);
    if (lane == 31) scratch[warp] = y;
    __syncthreads();
    static_assert(kPlanThreads == 32 * 32, "one warp's sum a lane");
    const Three w = warp_scan3(scratch[lane]);       // every warp adds up the warps' sums
    all = lane_of(w, 31);
    Three before = lane_of(w, max(warp - 1, 0));
    if (warp == 0) before = Three{0, 0, 0};
    return Three{before.back + y.back - x.back, before.need + y.need - x.need, before.tok + y.tok - x.tok};
}

// One sequence's wishes: pages to put back, pages to take, new tokens.
struct Wish {
    int32_t len, held, add;
    int32_t back, need, tok;
    bool ended, fits;
};

__device__ __forceinline__ Wish wish_of(const PagedReserveArgs& a, int32_t b, bool& bad) {
    Wish w;
    const int32_t most = a.max_pages << a.shift, page = 1 << a.shift;
    w.add = a.add[b];
    w.len = a.lens[b];
    if (w.len < 0 || w.len > most) {
        bad = true;
        w.len = max(0, min(w.len, most));
    }
    w.held = (w.len + page - 1) >> a.shift;
    w.ended = w.add < 0;
    w.back = w.ended ? w.held : 0;
    w.tok = max(w.add, 0);
    w.fits = !w.ended && w.tok <= most - w.len;
    w.need = w.fits ? (int32_t)(((int64_t)w.len + w.tok + page - 1) >> a.shift) - w.held : 0;
    return w;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const PagedReserveArgs a, const int32_t here) {
    __shared__ Three scratch[kPlanThreads / 32];
    __shared__ PagedSeq kept[kPlanSeqs];
    __shared__ int32_t kept_back[kPlanSeqs];
    grid_wait();
    grid_go();
    const int tid = threadIdx.x;
    const bool small = a.B <= kPlanSeqs;
    PagedSeq* seqs = small ? kept : a.seqs;
    int32_t* backs = small ? kept_back : a.back;
    const int32_t per = (a.B + kPlanThreads - 1) / kPlanThreads;
    const int32_t b0 = min((int64_t)tid * per, (int64_t)a.B), b1 = min((int64_t)b0 + per, (int64_t)a.B);
    const int32_t n0_given = *a.n_free, n0 = max(0, min(n0_given, a.pages));
    bool bad = n0 != n0_given, full = false;
    Three mine{0, 0, 0}, all;
    Wish w{};
    for (int32_t b = b0; b < b1; ++b) {
        w = wish_of(a, b, bad);
        mine.back += w.back;
        mine.need += w.need;
        mine.tok += w.tok;
    }
    Three at = scan3(mine, all, scratch);
    // more pages than the stack holds would be one put back twice
    const int32_t n1 = (int32_t)min((int64_t)n0 + all.back, (int64_t)a.pages);
    bad = bad || n0 + all.back > a.pages;
    int64_t taken = 0;
    for (int32_t b = b0; b < b1; ++b) {
        if (per > 1) w = wish_of(a, b, bad);
        const bool room = w.need == 0 || at.need + w.need <= n1, in_call = at.tok + w.tok <= a.T;
        const bool served = w.fits && room && in_call;
        if (w.tok > 0 && !served) {
            if (in_call) full = true; else bad = true;
        }
        PagedSeq q;
        q.tok = (int32_t)min(at.tok, (int64_t)a.T);
        q.len = w.len;
        q.held = served ? w.held : -1;
        // n1 - 1 - at.need is below zero only where nothing is taken
        q.top = (int32_t)(served && w.need ? n1 - 1 - at.need + w.held : 0);
        seqs[b] = q;
        if (!small || here < 0) a.seqs[b] = q;
        backs[b] = (int32_t)min(at.back, (int64_t)a.pages);
        a.cu[b] = q.tok;
        a.lens_out[b] = w.ended ? 0 : served ? w.len + w.tok : w.len;
        if (served) taken += w.need;
        at.back += w.back;
        at.need += w.need;
        at.tok += w.tok;
    }
    const int32_t total = (int32_t)min(all.tok, (int64_t)a.T);
    if (bad) set_error(a.status, ATTN_E_BOUNDS);
    if (full) set_error(a.status, ATTN_E_CAPACITY);
    // pages taken by all
    for (int m = 16; m > 0; m >>= 1) taken += __shfl_xor_sync(0xffffffffu, taken, m);
    __syncthreads();                                 // scratch is read, the records are written
    if ((tid & 31) == 0) scratch[tid >> 5].need = taken;
    // ended sequences' pages go onto the stack, in order: one thread a page
    const int32_t put = n1 - n0;
    for (int32_t i = tid; i < put; i += kPlanThreads) {
        int32_t lo = 0, hi = a.B;                    // the last sequence with at most i pages before it
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) >> 1;
            if (backs[mid] <= i) lo = mid; else hi = mid;
        }
        a.free_pages[n0 + i] = a.table[(int64_t)lo * a.table_ld + (i - backs[lo])];
    }
    __syncthreads();
    if (tid == 0) {
        int64_t sum = 0;
        for (int i = 0; i < kPlanThreads / 32; ++i) sum += scratch[i].need;
        *a.n_free_out = (int32_t)(n1 - sum);
        a.cu[a.B] = total;
    }
    if (here >= 0)
        for (int32_t t = tid; t < here; t += kPlanThreads) a.slots[t] = slot_of(a, seqs, total, t);
}

__global__ void __launch_bounds__(kSlotThreads) slots_kernel(const PagedReserveArgs a) {
    grid_wait();
    grid_go();
    const int32_t total = a.cu[a.B];
    for (int64_t t = (int64_t)blockIdx.x * kSlotThreads + threadIdx.x; t < a.T; t += (int64_t)gridDim.x * kSlotThreads)
        a.slots[t] = slot_of(a, a.seqs, total, (int32_t)t);
}

// ------------------------------------------------------------------ store

constexpr int kRowThreads = 256;
constexpr int kAtOnce = 4;               // pieces of K, and as many of V, that a thread has in flight

__global__ void __launch_bounds__(kRowThreads) store_kernel(const PagedStoreArgs a) {
    grid_wait();
    grid_go();
    const int64_t first = (int64_t)blockIdx.x * (kRowThreads * kAtOnce) + threadIdx.x;
    uint4 k[kAtOnce], v[kAtOnce];
    int64_t to[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
        const int64_t e = first + u * kRowThreads;
        to[u] = -1;
        if (e >= a.pieces) continue;
        const uint32_t row = a.by_vec.div((uint32_t)e), x = (uint32_t)e - row * a.by_vec.d;
        const uint32_t t = a.by_h.div(row), h = row - t * a.by_h.d;
        const int32_t slot = a.slots[t];
        if (slot == -1) continue;
        if (slot < 0 || (slot >> a.c.shift) >= a.c.pages) {
            set_error(a.status, ATTN_E_BOUNDS);
            continue;
        }
        const int64_t from = t * a.st + h * a.sh + 8 * (int64_t)x;
        to[u] = (slot >> a.c.shift) * a.c.sp + (slot & ((1 << a.c.shift) - 1)) * a.c.st + h * a.c.sh + 8 * (int64_t)x;
        k[u] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.k) + from));
        v[u] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + from));
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
        if (to[u] >= 0) {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.c.k) + to[u]) = k[u];
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.c.v) + to[u]) = v[u];
        }
}

}  // namespace

cudaError_t launch_paged_reserve(const PagedReserveArgs& a, cudaStream_t s) {
    const bool one = a.T <= kInlineTokens;
    cudaError_t e = launch_early(reserve_kernel, dim3(1), kPlanThreads, 0, 1, s, a, one ? a.T : -1);
    if (e != cudaSuccess || one) return e;
    const int blocks = std::min((a.T - 1) / kSlotThreads + 1, 8 * device_sm_count());
    return launch_early(slots_kernel, dim3(blocks), kSlotThreads, 0, 1, s, a);
}

cudaError_t launch_paged_store(const PagedStoreArgs& a, cudaStream_t s) {
    const int per = kRowThreads * kAtOnce;
    return launch_early(store_kernel, dim3((unsigned)(((int64_t)a.pieces + per - 1) / per)), kRowThreads, 0, 1, s, a);
}

}  // namespace attn
