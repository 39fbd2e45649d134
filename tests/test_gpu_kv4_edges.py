"""GPU tests of the 4-bit cache and of the key mass where test_gpu_kv4.py has none: rows
without a log-sum-exp whose queries are not finite, keys that are not, calls of several
threads at once, weights of more rows than one pass takes, buffers of weights used again,
caches within one allocation, the kernels that large shapes pick, slots behind the last one
that hold NaN, forked captures.
Tolerances are those derived there."""
import ctypes
import math
import os
import re
import threading

import numpy as np
import pytest
import torch

import chunked_causal_attention_gb300 as cca
from chunked_causal_attention_gb300 import _lib

from oracle import kv4 as K

from test_gpu_kv4 import (MASSES, MASS_PLANS, SUM, bf16, built, cached, check_attend, check_mass, f64, i32, random_cache,
                          score_error)

pytestmark = pytest.mark.gpu

NOT_FINITE = (float("nan"), float("inf"), -float("inf"))


def unset_rows(q, rows):
    """A copy of q [B, H, T, D] whose given rows hold NaN, infinities or the largest values."""
    q = q.clone()
    for i, t in enumerate(rows):
        q[:, i % q.shape[1], t] = (NOT_FINITE + (3e38, -3e38))[i % 5]
        q[:, i % q.shape[1], t, i % 8] = NOT_FINITE[i % 3]
    return q


# ------------------------------------------------------------------ key mass: rows without a log-sum-exp

@pytest.mark.parametrize("plan", ["whole", "cut", "docs", "late context"])
@pytest.mark.parametrize("D,H,Hkv", [(128, 4, 4), (64, 6, 2), (80, 4, 1), (256, 2, 1)])
def test_key_mass_of_rows_without_lse_that_are_not_finite(plan, D, H, Hkv):
    """Such rows count for nothing, as if their queries were any others: the same bits."""
    rng = np.random.default_rng(D + H)
    L, chunks = 700, MASS_PLANS[plan]
    q, k = 2 * bf16(rng, 2, H, L, D), bf16(rng, 2, Hkv, L, D)
    _, lse = cca.forward(q, k, k, chunks)
    rows = [3, 127, 128, 130, 255, 300, 301, 444, 445, 446, 511, 512, 640, 699]
    for i, t in enumerate(rows):
        lse[:, i % H, t] = -math.inf
    ws = cca.key_mass_workspace(q, k, chunks)
    want = cca.key_mass(q, k, lse, chunks, ws=ws)
    check_mass(q, k, lse, chunks, want, D ** -0.5)
    got = cca.key_mass(unset_rows(q, rows), k, lse, chunks, ws=ws)
    assert cca.attn_status(ws) == 0 and torch.equal(got, want)


def test_key_mass_after_a_forward_over_a_nan_query():
    """The forward gives a NaN query row the log-sum-exp -inf; the other rows' weights stand."""
    rng = np.random.default_rng(7)
    q, k = 2 * bf16(rng, 1, 2, 900, 128), bf16(rng, 1, 1, 900, 128)
    chunks = cca.attn_plan(900, 2, cca.PLAN_FLOPS)
    bad = q.clone()
    bad[0, 0, 650] = float("nan")
    _, lse = cca.forward(bad, k, k, chunks)
    assert lse[0, 0, 650] == -math.inf and int(lse.isfinite().sum()) == 2 * 900 - 1
    check_mass(q, k, lse, chunks, cca.key_mass(bad, k, lse, chunks), 128 ** -0.5)


def log_sum_exps(q, k, chunks, scale):
    """lse [B, H, T] of the chunks' rows in 64 bits, rounded once (zero elsewhere)."""
    B, H, T, _ = q.shape
    lse = torch.zeros(B, H, T, device="cuda")
    for a, b, ctx, _ in chunks:
        t = torch.arange(a, b, device="cuda")[:, None]
        seen = torch.arange(ctx, b, device="cuda")[None, :] <= t
        for h in range(H):
            s = q[:, h, a:b].double() @ k[:, h * k.shape[1] // H, ctx:b].double().transpose(-1, -2) * scale
            lse[:, h, a:b] = torch.logsumexp(s.masked_fill(~seen, -math.inf), -1)
    return lse


# rows of all heads of a group (w * H / Hkv): 200, 250 (a half of 64 columns ends in rows past the last), 15, 128, 300, 1
WINDOWS = [(128, 4, 1, 50), (64, 10, 2, 50), (80, 3, 1, 5), (256, 2, 1, 64), (40, 6, 2, 100), (128, 2, 2, 1)]


@pytest.mark.parametrize("D,H,Hkv,w", WINDOWS)
def test_key_mass_of_a_window_with_rows_without_lse_that_are_not_finite(D, H, Hkv, w):
    rng = np.random.default_rng(D + w)
    L = 3001
    q, k = 2 * bf16(rng, 2, H, L, D), bf16(rng, 2, Hkv, L, D)
    chunks = [(L - w - 3, L - 3, 7, 0)]
    lse = log_sum_exps(q, k, chunks, D ** -0.5)
    rows = [L - 4 - i for i in range(0, w, 7)]
    for i, t in enumerate(rows):
        lse[:, i % H, t] = -math.inf
    want = cca.key_mass(q, k, lse, chunks)
    check_mass(q, k, lse, chunks, want, D ** -0.5)
    assert torch.equal(cca.key_mass(unset_rows(q, rows), k, lse, chunks), want)


@pytest.mark.parametrize("D,H,Hkv,w", WINDOWS)
@pytest.mark.parametrize("pieces", [1, 2])
def test_key_mass_of_keys_that_are_not_finite(D, H, Hkv, w, pieces):
    """A key's infinity or NaN is its own: -inf scores weigh 0, +inf ones inf, NaN ones NaN, whichever kernel
    the number of chunks picks, and the other keys' weights stay."""
    rng = np.random.default_rng(3 * D + w)
    L, scale = 3001, D ** -0.5
    q, k = 2 * bf16(rng, 1, H, L, D), bf16(rng, 1, Hkv, L, D)
    q[..., 0] = q[..., 0].abs() + 0.25
    low, high, nan = [0, 5, 130, 1000, 2047, 2 * L // 3], [6, 131, 1001], [9, 1002]
    w = max(w, pieces)
    cut = L - w + w // 2
    chunks = [(L - w, L, 0, 0)] if pieces == 1 else [(L - w, cut, 0, 0), (cut, L, 0, 0)]
    lse = log_sum_exps(q, k, chunks, scale)
    want = cca.key_mass(q, k, lse, chunks)
    check_mass(q, k, lse, chunks, want, scale)
    bad = k.clone()
    bad[:, :, low, 0], bad[:, :, high, 0], bad[:, :, nan, D - 1] = -math.inf, math.inf, math.nan
    got = cca.key_mass(q, bad, lse, chunks)
    assert (got[..., low] == 0).all() and (got[..., high] == math.inf).all() and got[..., nan].isnan().all()
    other = torch.ones(L, dtype=torch.bool)
    other[low + high + nan] = False
    assert torch.equal(got[..., other], want[..., other])


# D, query and key/value heads, batch, rows, keys: long enough for the kernel of few rows over many keys
LONG = [(128, 32, 8, 1, 1, 16384), (128, 8, 8, 1, 100, 40007), (64, 40, 8, 1, 50, 40000), (80, 24, 8, 1, 5, 16384),
        (256, 16, 8, 2, 60, 20000), (40, 64, 8, 1, 60, 30001), (64, 8, 1, 3, 33, 120000), (128, 24, 3, 1, 40, 100001)]


def window_call(*a, **kw):
    """key_mass, as the kernel of few rows takes it: one launch, where the general one uploads its lists."""
    launches = cca.kernel_launches()
    out = cca.key_mass(*a, **kw)
    assert cca.kernel_launches() - launches == 1
    return out


def check_rows(q, k, lse, chunk, got, scale, heads, mass_in=None):
    """check_mass of one chunk for some key/value heads, with errors from the chunk's rows alone (all rows against
    all keys of a long prompt would not fit)."""
    a, b, ctx, _ = chunk
    G = q.shape[1] // k.shape[1]
    for i in range(q.shape[0]):
        for hk in heads:
            qs, ls, kh = f64(q[i, hk * G:hk * G + G]), f64(lse[i, hk * G:hk * G + G]), f64(k[i, hk])
            ref, rows = K.key_mass(qs, kh, ls, [chunk], scale), ls[:, a:b]
            e = score_error(qs[:, a:b].reshape(-1, qs.shape[-1]), kh[ctx:b], scale) + 2.0 ** -22 * np.abs(rows[np.isfinite(rows)]).max()
            base = f64(mass_in[i, hk]) if mass_in is not None else 0.0
            tol = (2 * e + SUM) * ref + 2.0 ** -22 * np.abs(base + ref) + 1e-35
            assert (np.abs(f64(got[i, hk]) - base - ref) <= tol).all()


@pytest.mark.parametrize("D,H,Hkv,B,w,T", LONG)
def test_key_mass_of_few_rows_over_many_keys(D, H, Hkv, B, w, T):
    rng = np.random.default_rng(D + w)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    scale, heads = D ** -0.5, sorted({0, Hkv - 1})
    q = 2 * torch.randn(B, H, T, D, device="cuda", generator=g).bfloat16()
    k = torch.randn(B, Hkv, T, D, device="cuda", generator=g).bfloat16()
    q[..., 0] = q[..., 0].abs() + 0.25
    chunks = [(T - w - 3, T - 3, 300, 0)]                            # the first and last keys are seen by no row
    lse = log_sum_exps(q, k, chunks, scale)
    lse[:, 0, T - 4] = -math.inf                                     # a row that counts for nothing
    ws = cca.key_mass_workspace(q, k, chunks)
    want = window_call(q, k, lse, chunks, ws=ws)
    check_rows(q, k, lse, chunks[0], want, scale, heads)
    assert (want[..., :300] == 0).all() and (want[..., T - 3:] == 0).all()
    m = torch.rand(B, Hkv, T, device="cuda")
    start = m.clone()
    window_call(q, k, lse, chunks, mass_in=m, mass_out=m, ws=ws)
    check_rows(q, k, lse, chunks[0], m, scale, heads, mass_in=start)
    for _ in range(3):
        assert torch.equal(window_call(q, k, lse, chunks, ws=ws), want)
    # rows without a log-sum-exp that hold anything
    rows = [T - 4 - i for i in range(0, w, 7)]
    for i, t in enumerate(rows):
        lse[:, i % H, t] = -math.inf
    some = window_call(q, k, lse, chunks, ws=ws)
    assert torch.equal(window_call(unset_rows(q, rows), k, lse, chunks, ws=ws), some)
    check_rows(q, k, lse, chunks[0], some, scale, heads)
    # keys that are not finite
    low, high, nan = [300, 305, 1000, T // 2], [306, 1001], [309, 1002]
    bad = k.clone()
    bad[:, :, low, 0], bad[:, :, high, 0], bad[:, :, nan, D - 1] = -math.inf, math.inf, math.nan
    lse = log_sum_exps(q, k, chunks, scale)
    want, got = (window_call(q, x, lse, chunks, ws=ws) for x in (k, bad))
    assert (got[..., low] == 0).all() and (got[..., high] == math.inf).all() and got[..., nan].isnan().all()
    other = torch.ones(T, dtype=torch.bool)
    other[low + high + nan] = False
    assert torch.equal(got[..., other], want[..., other]) and cca.attn_status(ws) == 0


def test_waits_of_the_kernel_of_few_rows_run_out(monkeypatch):
    rng = np.random.default_rng(71)
    q, k, chunks = bf16(rng, 1, 32, 16384, 64), bf16(rng, 1, 8, 16384, 64), [(16380, 16384, 0, 0)]
    lse, ws = log_sum_exps(q, k, chunks, 0.125), cca.key_mass_workspace(q, k, chunks)
    want = window_call(q, k, lse, chunks, ws=ws)
    monkeypatch.setenv("ATTN_TEST_STALL_PRODUCER", "1")
    monkeypatch.setenv("ATTN_WAIT_LIMIT_MS", "200")
    window_call(q, k, lse, chunks, ws=ws)
    assert cca.attn_status(ws) == 6
    monkeypatch.delenv("ATTN_TEST_STALL_PRODUCER")
    assert torch.equal(window_call(q, k, lse, chunks, ws=ws), want) and cca.attn_status(ws) == 0


@pytest.mark.parametrize("D,H,Hkv,w,T,one", [
    (128, 32, 8, 1, 16384, True), (128, 32, 8, 64, 131072, True), (128, 32, 8, 64, 2048, False), (128, 32, 8, 128, 16384, False),
    (64, 32, 8, 256, 16384, False), (128, 8, 8, 128, 2048, False), (128, 8, 8, 128, 65536, True), (256, 8, 8, 128, 2048, False)])
def test_which_kernel_takes_a_window(D, H, Hkv, w, T, one):
    """By the tiles of keys that an SM takes: below, the general kernel is up to five times as fast."""
    q, k = torch.zeros(1, H, T, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, Hkv, T, D, dtype=torch.bfloat16, device="cuda")
    chunks, lse = [(T - w, T, 0, 0)], torch.zeros(1, H, T, device="cuda")
    ws, launches = cca.key_mass_workspace(q, k, chunks), cca.kernel_launches()
    cca.key_mass(q, k, lse, chunks, ws=ws)
    assert (cca.kernel_launches() - launches == 1) == one


# ------------------------------------------------------------------ calls of several threads at once

def at_once(*calls, times):
    """Each call (of a stream's handle, returning a status) many times in a thread of its own, on a stream of its
    own; the statuses that are not ATTN_OK."""
    bad, start = [], threading.Barrier(len(calls))
    torch.cuda.synchronize()

    def work(call, stream):
        start.wait()
        for _ in range(times):
            status = call(stream.cuda_stream)
            if status:
                bad.append(status)

    threads = [threading.Thread(target=work, args=(c, torch.cuda.Stream())) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return bad


def test_evictions_of_two_threads():
    """Caches of different capacity ask for different amounts of shared memory in the same kernel. The C calls
    themselves, on short sequences, so that the threads are in them most of the time."""
    calls, results, fn = [], [], cca.lib().attn_kv4_evict
    for cap in (300000, 90000):
        src, dst = random_cache(1, 1, cap, 8, cap), cca.kv4_cache(1, 1, 512, 8, k_scale=0.5, v_scale=2.0)
        mass, lens, out = torch.rand(1, 1, cap, device="cuda"), i32([600]), i32([0])
        slots, ws = torch.empty(1, 1, 500, dtype=torch.int32, device="cuda"), cca.kv4_workspace(src)
        want = cca.kv4_evict(src, lens, mass, 500, 3, dst)[1]
        args = (ctypes.byref(src.desc), lens.data_ptr(), mass.data_ptr(), cap, 500, 3, ctypes.byref(dst.desc),
                out.data_ptr(), None, 0, slots.data_ptr(), ws.data_ptr(), ws.numel())
        calls.append(lambda s, a=args: fn(*a, s))
        results.append((slots, want, ws, src, dst, mass, lens, out))       # args holds addresses only
    assert at_once(*calls, times=20000) == []
    for slots, want, ws, *_ in results:
        assert torch.equal(slots, want) and cca.attn_status(ws) == 0


def test_window_masses_of_two_threads():
    """Windows of different length ask for different amounts of shared memory in the same kernel."""
    calls, results, fn = [], [], cca.lib().attn_key_mass
    for w in (1, 32):
        rng = np.random.default_rng(w)
        q, k = bf16(rng, 1, 64, 8192, 64), bf16(rng, 1, 8, 8192, 64)
        chunks = [(8192 - w, 8192, 0, 0)]
        lse = log_sum_exps(q, k, chunks, 0.125)
        ws, shape, out = cca.key_mass_workspace(q, k, chunks), cca.shape_of(q, None, False, k), torch.zeros(1, 8, 8192, device="cuda")
        want = window_call(q, k, lse, chunks, ws=ws)
        arr, n = _lib.chunk_array(chunks)
        args = (q.data_ptr(), k.data_ptr(), lse.data_ptr(), arr, n, ctypes.byref(shape), None, out.data_ptr(),
                ws.data_ptr(), ws.numel())
        calls.append(lambda s, a=args: fn(*a, s))
        results.append((out, want, ws, q, k, lse, shape))
    assert at_once(*calls, times=20000) == []
    for out, want, ws, *_ in results:
        assert torch.equal(out, want) and cca.attn_status(ws) == 0


def test_merges_of_two_threads():
    """Forwards with re-split chunks at 8 and 128 dims: the merge kernel is one, its shared memory is not."""
    calls, results, fn = [], [], cca.lib().attn_fwd
    for D in (8, 128):
        q = bf16(np.random.default_rng(D), 1, 1, 2048, D)
        chunks = [(0, 1920, 0, 0), (1920, 2048, 0, -4)]
        shape, o, lse = cca.shape_of(q), torch.zeros_like(q), torch.zeros(1, 1, 2048, device="cuda")
        ws = cca.workspace(shape, chunks, cca.PASS_FWD)
        want = cca.forward(q, q, q, chunks)
        arr, n = _lib.chunk_array(chunks)
        args = (q.data_ptr(), q.data_ptr(), q.data_ptr(), arr, n, ctypes.byref(shape), o.data_ptr(), lse.data_ptr(),
                ws.data_ptr(), ws.numel())
        calls.append(lambda s, a=args: fn(*a, s))
        results.append((o, lse, want, ws, q, shape))
    assert at_once(*calls, times=20000) == []
    for o, lse, want, ws, *_ in results:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and cca.attn_status(ws) == 0


# ------------------------------------------------------------------ attention of many rows

def mostly_empty_cache(B, Hkv, cap, D, used, seed):
    """A cache whose first `used` slots are random and whose others hold NaN scales."""
    c, near = cca.kv4_cache(B, Hkv, cap, D, k_scale=0.5, v_scale=2.0), random_cache(B, Hkv, used, D, seed)
    for a, b in zip((c.k_codes, c.k_scales, c.v_codes, c.v_scales), (near.k_codes, near.k_scales, near.v_codes, near.v_scales)):
        a.fill_(0x7F)
        a[:, :, :used] = b
    return c


def nan_behind(c, lens):
    for b, n in enumerate(lens):
        c.k_scales[b, :, n:], c.v_scales[b, :, n:] = 0x7F, 0xFF


@pytest.mark.parametrize("B,cap,H,T,D,lens", [
    (1, 1 << 20, 2, 150, 8, [700]),                       # 10 groups of 32 rows in two passes
    (2, 1 << 20, 3, 101, 40, [900, 77]),                  # 303 rows in three; the first rows of a sequence see nothing
    (1, (1 << 20) - 16, 1, 300, 8, [513]),                # 38 groups of 8 rows in two
    (1, 1 << 20, 1, 300, 136, [600])])                    # 19 groups of 16 rows in two
def test_weights_of_more_rows_than_one_pass_takes(B, cap, H, T, D, lens):
    rng = np.random.default_rng(D + T)
    c = mostly_empty_cache(B, 1, cap, D, 1024, T)
    q = 2 * bf16(rng, B, H, T, D)
    ws = cca.kv4_workspace(c, q, mass=True)
    rows = -(-H * T // 8) * 8
    assert ws.numel() < 4 * B * cap * rows                # the scores of all rows at once would be this
    mi, mo = torch.rand(B, 1, cap, device="cuda"), torch.full((B, 1, cap), -3.0, device="cuda")
    launches = cca.kernel_launches()
    o, lse = cca.kv4_attention(q, c, i32(lens), mass_in=mi, mass_out=mo, ws=ws)
    assert cca.kernel_launches() - launches >= 6
    check_attend(q, c, lens, o, lse, None, mi, mo, kept_tail=-3.0)
    m = mi.clone()
    cca.kv4_attention(q, c, i32(lens), mass_in=m, mass_out=m, ws=ws)
    for b, n in enumerate(lens):
        assert torch.equal(m[b, :, :n], mo[b, :, :n]) and torch.equal(m[b, :, n:], mi[b, :, n:])
    cca.kv4_attention(q, c, i32(lens), mass_out=mo, ws=ws)
    check_attend(q, c, lens, o, lse, None, None, mo, kept_tail=-3.0)
    assert cca.attn_status(ws) == 0


def groups_of_32_rows(c, q):
    """Whether the call of these shapes runs on groups of 32 rows: the scores in its workspace say so."""
    rows = q.shape[1] // c.Hkv * q.shape[2]
    more = cca.kv4_workspace(c, q, mass=True).numel() - cca.kv4_workspace(c, q).numel()
    return more >= 4 * c.B * c.Hkv * c.cap * 32 * -(-rows // 32)


@pytest.mark.parametrize("D", [40, 64, 80, 128])
@pytest.mark.parametrize("G,T", [(32, 1), (11, 3), (4, 16), (1, 40)])
def test_attend_with_four_groups_of_rows(D, G, T):
    """At least 32 rows a head and 2^20 slots: the kernels that take 32 rows at a time (33 and 40 rows: the last
    group nearly empty)."""
    B, Hkv, cap = 2, 2, 262144
    lens = [6, 4999] if T > 1 else [0, 4999]
    c = mostly_empty_cache(B, Hkv, cap, D, 5008, D + G)
    nan_behind(c, lens)
    q = 2 * bf16(np.random.default_rng(D + 7 * G + T), B, Hkv * G, T, D)
    assert B * Hkv * cap >= 1 << 20 and G * T >= 32 and groups_of_32_rows(c, q)
    ws = cca.kv4_workspace(c, q, mass=True)
    o, lse = cca.kv4_attention(q, c, i32(lens), ws=ws)
    check_attend(q, c, lens, o, lse)
    mi, mo = torch.rand(B, Hkv, cap, device="cuda"), torch.full((B, Hkv, cap), -3.0, device="cuda")
    o2, lse2 = cca.kv4_attention(q, c, i32(lens), mass_in=mi, mass_out=mo, ws=ws)
    check_attend(q, c, lens, o2, lse2, None, mi, mo, kept_tail=-3.0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and cca.attn_status(ws) == 0
    for _ in range(3):
        again = torch.full_like(mo, -3.0)
        o2, lse2 = cca.kv4_attention(q, c, i32(lens), mass_in=mi, mass_out=again, ws=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(mo, again)


@pytest.mark.parametrize("D", [40, 64, 80, 128])
@pytest.mark.parametrize("what", ["k", "v"])
def test_attend_nan_rows_with_four_groups_of_rows(D, what):
    """A NaN slot among those in use reaches the queries that see it and no other."""
    T, n, cap = 20, 3150, 1 << 20
    c = mostly_empty_cache(1, 1, cap, D, 3200, D)
    blk = -(-D // 16) // 2
    getattr(c, what + "_scales")[0, 0, n - 2, blk] = 0x7F          # seen by queries T-2 and T-1
    q = bf16(np.random.default_rng(13), 1, 2, T, D)
    assert groups_of_32_rows(c, q)
    o, lse = cca.kv4_attention(q, c, i32([n]))
    bad = o[0, :, T - 2:].isnan()
    if what == "k":
        assert bad.all() and lse[0, :, T - 2:].isnan().all()
    else:
        hit = torch.zeros(D, dtype=torch.bool, device="cuda")
        hit[16 * blk:16 * blk + 16] = True
        assert (bad == hit).all() and lse.isfinite().all()
    assert o[0, :, :T - 2].isfinite().all() and lse[0, :, :T - 2].isfinite().all()


@pytest.mark.parametrize("D", [64, 72, 128, 256])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000, 4095, 4096])
def test_attend_lengths_with_nan_behind(D, n):
    c = random_cache(1, 3, 4096, D, n)
    nan_behind(c, [n])
    q = 2 * bf16(np.random.default_rng(n), 1, 12, 2, D)
    mo = torch.zeros(1, 3, 4096, device="cuda")
    o, lse = cca.kv4_attention(q, c, i32([n]), mass_out=mo)
    check_attend(q, c, [n], o, lse, None, None, mo, kept_tail=0.0)


def test_attend_ragged_with_nan_behind():
    rng = np.random.default_rng(61)
    lens = [int(x) for x in rng.integers(0, 500, 70)]
    c = random_cache(70, 2, 512, 128, 62)
    nan_behind(c, lens)
    q = bf16(rng, 70, 10, 3, 128)
    o, lse = cca.kv4_attention(q, c, i32(lens))
    check_attend(q, c, lens, o, lse)


def test_attend_in_a_captured_fork():
    """Two attentions on forked streams of one capture, joined by an eviction; replayed with other lengths."""
    rng = np.random.default_rng(63)
    B, Hkv, cap, D = 2, 2, 2048, 128
    c, d = random_cache(B, Hkv, cap, D, 64), random_cache(B, Hkv, cap, D, 65)
    small = cca.kv4_cache(B, Hkv, 256, D, k_scale=0.5, v_scale=2.0)
    q, lens = [bf16(rng, B, 8, t, D) for t in (1, 5)], i32([2000, 300])
    mass, kept, out = torch.rand(B, Hkv, cap, device="cuda"), torch.zeros(B, Hkv, 256, device="cuda"), i32([0, 0])
    ws = [cca.kv4_workspace(c, q[0], mass=True), cca.kv4_workspace(d, q[1])]
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        lens.add_(1)
        side.wait_stream(here)
        with torch.cuda.stream(side):
            o1, l1 = cca.kv4_attention(q[1], d, lens, ws=ws[1])
        o0, l0 = cca.kv4_attention(q[0], c, lens, mass_in=mass, mass_out=mass, ws=ws[0])
        here.wait_stream(side)
        _, slots = cca.kv4_evict(c, lens, mass, 200, 8, small, kept, lens_out=out, ws=ws[0])
        o2, l2 = cca.kv4_attention(q[0], small, out, ws=ws[0])
    for start in ([2000, 300], [7, 2047], [0, 1]):
        lens.copy_(i32(start))
        m = mass.clone()
        graph.replay()
        n = i32([x + 1 for x in start])
        e0, f0 = cca.kv4_attention(q[0], c, n, mass_in=m, mass_out=m)
        e1, f1 = cca.kv4_attention(q[1], d, n)
        small2, kept2 = cca.kv4_cache(B, Hkv, 256, D, k_scale=0.5, v_scale=2.0), torch.zeros_like(kept)
        n2, s2 = cca.kv4_evict(c, n, m, 200, 8, small2, kept2)
        e2, f2 = cca.kv4_attention(q[0], small2, n2)
        for x, y in ((o0, e0), (l0, f0), (o1, e1), (l1, f1), (o2, e2), (l2, f2), (slots, s2), (mass, m), (out, n2)):
            assert torch.equal(x, y)
    assert cca.attn_status(ws[0]) == 0 and cca.attn_status(ws[1]) == 0


# ------------------------------------------------------------------ buffers of weights used again

def test_the_serving_example_with_a_buffer_in_use_before():
    """README's example as it stands, into a cache and weights that held something else: the token that it
    appends starts from no weight."""
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    example, = (b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "kv4_evict(" in b)
    rng = np.random.default_rng(51)
    B, H, Hkv, D, L, keep = 1, 2, 1, 64, 5000, 4096
    g = {"cca": cca, "B": B, "Hkv": Hkv, "D": D, "L": L, "cap": 5008, "T": 16, "pos": i32([0]), "lens": i32([L])}
    g["q"], g["k"], g["v"] = 2 * bf16(rng, B, H, L, D), bf16(rng, B, Hkv, L, D), bf16(rng, B, Hkv, L, D)
    g["chunks"] = cca.attn_plan(L, 2, cca.PLAN_FLOPS)
    _, g["lse"] = cca.forward(g["q"], g["k"], g["v"], g["chunks"])
    g["small"], g["mass2"] = random_cache(B, Hkv, 4112, D, 52, ts=(1.0, 1.0)), torch.full((B, Hkv, 4112), 9.0, device="cuda")
    g["q1"], g["k1"], g["v1"] = bf16(rng, B, H, 1, D), bf16(rng, B, Hkv, 1, D), bf16(rng, B, Hkv, 1, D)
    g["ws"] = cca.kv4_workspace(g["small"], g["q1"], mass=True)
    exec(example, g)
    assert g["lens2"].tolist() == [keep + 1] and cca.attn_status(g["ws"]) == 0
    before = torch.zeros(B, Hkv, 4112, device="cuda")
    before[..., :keep] = g["mass"].gather(2, g["slots"].long())
    check_attend(g["q1"], g["small"], [keep + 1], g["o"], g["lse1"], None, before, g["mass2"])


def test_two_caches_in_turn():
    """Decoding and eviction over and over between two caches and two buffers of weights: every slot's weight
    is that of its own token, and the slots are chosen by it."""
    rng = np.random.default_rng(53)
    B, H, Hkv, D, cap, keep, recent, steps = 2, 4, 2, 64, 128, 48, 8, 20
    caches = [random_cache(B, Hkv, cap, D, 54 + i) for i in range(2)]
    masses = [torch.full((B, Hkv, cap), 7.0 + i, device="cuda") for i in range(2)]
    lens = i32([100, 30])
    masses[0].copy_(torch.rand(B, Hkv, cap))
    masses[0][0, :, 100:], masses[0][1, :, 30:] = 0, 0
    true = f64(masses[0])
    ws = cca.kv4_workspace(caches[0], bf16(rng, B, H, 1, D), mass=True)
    for turn in range(4):
        a, b = turn % 2, 1 - turn % 2
        chosen = [[K.evict(masses[a][i, h].cpu().numpy(), int(lens[i]), keep, recent) for h in range(Hkv)] for i in range(B)]
        lens, slots = cca.kv4_evict(caches[a], lens, masses[a], keep, recent, caches[b], masses[b].zero_(), ws=ws)
        kept = np.zeros_like(true)
        for i in range(B):
            for h in range(Hkv):
                m = len(chosen[i][h])
                assert slots[i, h, :m].tolist() == chosen[i][h]
                kept[i, h, :m] = true[i, h, chosen[i][h]]
        true = kept
        for _ in range(steps):
            q, k, v = 2 * bf16(rng, B, H, 1, D), bf16(rng, B, Hkv, 1, D), bf16(rng, B, Hkv, 1, D)
            cca.kv4_store(caches[b], k, v, lens, ws=ws)
            lens += 1
            cca.kv4_attention(q, caches[b], lens, mass_in=masses[b], mass_out=masses[b], ws=ws)
            for i in range(B):
                for h in range(Hkv):
                    n = int(lens[i])
                    kk, vv = cached(caches[b], i, h, n)
                    true[i, h, :n] += K.attend(f64(q[i, 2 * h:2 * h + 2]), kk, vv, n, D ** -0.5)[2].sum((0, 1))
            # scores below 64 here: a weight is off by 2 (D + 4) 2^-23 64 + 2^-13 of itself at most (test_gpu_kv4)
            assert (np.abs(f64(masses[b]) - true) <= 2e-3 * true + 1e-30).all()
    assert cca.attn_status(ws) == 0


# ------------------------------------------------------------------ caches within one allocation

def test_evict_within_one_allocation():
    """From the front slots of a cache to slots behind them, heads between one another; and back."""
    rng = np.random.default_rng(57)
    B, Hkv, D, keep = 2, 3, 80, 100
    big = random_cache(B, Hkv, 640, D, 58)
    view = lambda a, b: cca.KV4Cache(*(t[:, :, a:b] for t in (big.k_codes, big.k_scales, big.v_codes, big.v_scales)), D=D,
                                     k_scale=big.k_scale, v_scale=big.v_scale)
    front, back, other = view(0, 512), view(512, 640), cca.kv4_cache(B, Hkv, 128, D, k_scale=0.5, v_scale=2.0)
    before = [t.clone() for t in (front.k_codes, front.v_scales)]
    mass, lens = torch.rand(B, Hkv, 512, device="cuda"), i32([512, 77])
    want = cca.kv4_evict(front, lens, mass, keep, 9, other)
    got = cca.kv4_evict(front, lens, mass, keep, 9, back)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for b, n in enumerate(want[0].tolist()):
        for x, y in ((back.k_codes, other.k_codes), (back.k_scales, other.k_scales), (back.v_codes, other.v_codes),
                     (back.v_scales, other.v_scales)):
            assert torch.equal(x[b, :, :n], y[b, :, :n])
    assert torch.equal(front.k_codes, before[0]) and torch.equal(front.v_scales, before[1])
    q = bf16(rng, B, 6, 1, D)
    for x, y in zip(cca.kv4_attention(q, back, got[0]), cca.kv4_attention(q, other, want[0])):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ eviction of many heads

def many_heads(B, Hkv):
    """As many heads as the eviction wants for one block of 512 threads a head."""
    return B * Hkv >= 2 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("kind", ["ties", "special"])
@pytest.mark.parametrize("keep,recent", [(2040, 0), (2056, 65), (2048, 2048), (300, 1)])
def test_evict_of_many_heads(kind, keep, recent):
    rng = np.random.default_rng(keep + recent)
    B, Hkv, cap, D = 48, 8, 4112, 64
    assert many_heads(B, Hkv)
    lens = [0, 1, keep, keep + 1, cap, 2047, 2048, 2049] + [int(x) for x in rng.integers(0, cap + 1, B - 8)]
    src = random_cache(B, Hkv, cap, D, 67)
    dst = cca.kv4_cache(B, Hkv, (keep + 15) // 16 * 16 + 16, D, k_scale=0.5, v_scale=2.0)
    for t in (dst.k_codes, dst.k_scales, dst.v_codes, dst.v_scales):
        t.fill_(0xCD)
    mass = torch.tensor(MASSES[kind](rng, (B, Hkv, cap)), dtype=torch.float32).cuda()
    mo, dl, ws = torch.full((B, Hkv, keep + 5), -7.0, device="cuda"), i32(lens), cca.kv4_workspace(src)
    _, slots = cca.kv4_evict(src, dl, mass, keep, recent, dst, mo, lens_out=dl, ws=ws)
    assert dl.tolist() == [min(n, keep) for n in lens] and cca.attn_status(ws) == 0
    hm, got = mass.cpu().numpy(), slots.cpu().numpy()
    for b, n in enumerate(lens):
        m = min(n, keep)
        for h in range(Hkv):
            assert got[b, h].tolist() == K.evict(hm[b, h], n, keep, recent) + [-1] * (keep - m)
        at = slots[b, :, :m, None].long()
        for a, z in ((src.k_codes, dst.k_codes), (src.k_scales, dst.k_scales), (src.v_codes, dst.v_codes),
                     (src.v_scales, dst.v_scales)):
            assert torch.equal(z[b, :, :m], a[b].gather(1, at.expand(-1, -1, a.shape[-1]))) and (z[b, :, m:] == 0xCD).all()
        assert torch.equal(mo[b, :, :m].view(torch.int32), mass[b].gather(1, at[..., 0]).view(torch.int32))
        assert (mo[b, :, m:] == -7).all()


@pytest.mark.parametrize("keep,recent", [(1000, 3), (32784, 0), (32790, 77)])
def test_evict_of_many_long_heads(keep, recent):
    """More slots than a block holds: the last ones' masses are read again for each pass."""
    rng = np.random.default_rng(keep)
    B, Hkv, cap, D = 48, 8, 32800 + 2048, 8
    assert many_heads(B, Hkv)
    lens = [cap, cap - 1, 32768, 32769, 5] + [int(x) for x in rng.integers(32000, cap + 1, B - 5)]
    src, dst = random_cache(B, Hkv, cap, D, 69), cca.kv4_cache(B, Hkv, (keep + 15) // 16 * 16, D, k_scale=0.5, v_scale=2.0)
    mass = torch.tensor(np.round(np.exp(rng.normal(size=(B, Hkv, cap))), 2), dtype=torch.float32).cuda()        # many ties
    _, slots = cca.kv4_evict(src, i32(lens), mass, keep, recent, dst)
    for b, n in enumerate(lens):
        m, r = min(n, keep), min(recent, n, keep)
        best = torch.sort(mass[b, :, :n - r], dim=-1, descending=True, stable=True).indices[:, :m - r]
        last = torch.arange(n - r, n, device="cuda").expand(Hkv, -1)
        assert torch.equal(slots[b, :, :m].long(), torch.cat((best.sort(-1).values, last), -1)) and (slots[b, :, m:] == -1).all()
        if b < 2:
            assert slots[b, 3, :m].tolist() == K.evict(mass[b, 3].cpu().numpy(), n, keep, recent)


# ------------------------------------------------------------------ layouts

@pytest.mark.parametrize("give", ["k", "v", "both", "neither"])
def test_load_into_a_view(give):
    """Rows into views of wider tensors, one of the two given or both."""
    c, pos = random_cache(2, 3, 64, 80, 73), i32([0, 30])
    wide = [torch.full((2, 20, 3, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = (w.permute(0, 2, 1, 3)[..., :80] for w in wide)
    want = cca.kv4_load(c, pos, 20)
    got = cca.kv4_load(c, pos, 20, k=k if give in ("k", "both") else None, v=v if give in ("v", "both") else None)
    for x, y in zip(got, want):
        assert torch.equal(x, y) and (give == "neither" or x.stride() == k.stride())
    for w in wide:
        assert (w[..., 80:] == 7).all()


@pytest.mark.parametrize("packed", [False, True])
def test_key_mass_of_few_rows_strided(packed):
    """Token-major storage of wider rows, as a batch view and as packed tokens, in the kernel of few rows."""
    g = torch.Generator(device="cuda")
    g.manual_seed(75)
    T, D, w, scale = 40010, 80, 20, 80 ** -0.5
    q = torch.randn(3, T, 16, 128, device="cuda", generator=g).bfloat16()[1:, ..., :D]
    k = torch.randn(3, T, 8, 96, device="cuda", generator=g).bfloat16()[1:, ..., :D]
    chunks = [(T - w - 5, T - 5, 11, 0)]
    qh, kh = (x.permute(0, 2, 1, 3) for x in (q, k))
    lse = log_sum_exps(qh, kh, chunks, scale)
    if packed:
        got = torch.cat([window_call(q[b], k[b], lse[b:b + 1], chunks, packed=True) for b in range(2)])
    else:
        got = window_call(qh, kh, lse, chunks)
    check_rows(qh, kh, lse, chunks[0], got, scale, [0, 7])
    assert torch.equal(got, window_call(qh.contiguous(), kh.contiguous(), lse, chunks))
