"""GPU parity of the paged key/value cache with the oracle (oracle.paged, oracle.kv4.attend).

Tolerances, derived from the arithmetic (relative errors of a rounding are half a step):
  * Tables, lengths, slots, stored rows: equal.
  * A score is a sum of D products of bf16 values, exact in fp32, each addition off by at
    most 2^-23 of the sum of magnitudes (a tensor core may truncate); scaling it and
    taking the maximum away round three times by 2^-24. With A the largest sum of
    magnitudes |q||k| |scale| of a head: e = (D + 4) 2^-23 A, and ex2.approx adds 2^-22. A sum
    of weights in fp32 has at most 2^10 terms in a partial sum: 2^10 2^-24.
  * A weight is rounded to bf16, 2^-8 of itself; parts are joined in fp32.
  * O is the weighted sum of |v| with those errors, rounded to bf16, 2^-8.
"""
import math
import os

import numpy as np
import pytest
import torch

import chunked_causal_attention_gb300 as cca
from oracle import kv4 as K
from oracle import paged as P

pytestmark = pytest.mark.gpu

SUM = 2.0 ** -14


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(cca._lib.LIB_PATH):
        from chunked_causal_attention_gb300 import build
        build.build()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(x):
    return x.detach().double().cpu().numpy()


def bf16(rng, *shape):
    return torch.tensor(rng.normal(size=shape), dtype=torch.float32).bfloat16().cuda()


def pool_of(rng, pages, Hkv, page, D, layout):
    """A pool full of NaN, seen as [pages, Hkv, page, D], in one of several orders and with gaps."""
    nan = lambda *s: torch.full(s, math.nan, dtype=torch.bfloat16, device="cuda")
    if layout == "heads":
        return [nan(pages, Hkv, page, D) for _ in range(2)]
    if layout == "slots":
        return [nan(pages, page, Hkv, D).transpose(1, 2) for _ in range(2)]
    if layout == "both":                                            # k and v of a slot next to each other
        kv = nan(pages, page, 2, Hkv, D)
        return [kv[:, :, i].transpose(1, 2) for i in range(2)]
    if layout == "gaps":
        return [nan(pages, Hkv + 1, page, D + 8)[:, 1:, :, :D] for _ in range(2)]
    return [nan(Hkv, pages, page, D).transpose(0, 1) for _ in range(2)]   # "outer": heads outside pages


class Batch:
    """Sequences over a pool of shuffled pages; slots behind the last one hold NaN."""

    def __init__(self, lens, nq, H, Hkv, D, page, layout="heads", seed=0, pad=0, extra=2, amp=2.0):
        rng = np.random.default_rng(seed)
        self.lens, self.nq, self.H, self.Hkv, self.D, self.page = lens, nq, H, Hkv, D, page
        held = [-(-n // page) for n in lens]
        pages = sum(held) + extra
        order = rng.permutation(pages)
        self.table = np.full((len(lens), max(held + [1]) + 1), -1)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.k, self.v = pool_of(rng, pages, Hkv, page, D, layout)
        for b, n in enumerate(lens):
            if not n:
                continue
            at = torch.as_tensor(self.table[b, :held[b]], device="cuda")
            for pool in (self.k, self.v):
                r = torch.full((held[b] * page, Hkv, D), math.nan, dtype=torch.bfloat16, device="cuda")
                r[:n] = bf16(rng, n, Hkv, D)
                pool[at] = r.view(held[b], page, Hkv, D).transpose(1, 2)
        self.cu = np.concatenate([[0], np.cumsum(nq)])
        self.T = int(self.cu[-1]) + pad
        self.q = (amp * bf16(rng, max(self.T, 1), H, D)).bfloat16()
        self.cache = cca.PagedCache(self.k, self.v)

    def want(self, scale=None):
        """(o, lse, bounds of |o| and of |lse|) by the oracle."""
        scale = self.D ** -0.5 if scale is None else scale
        o, lse = np.zeros((self.T, self.H, self.D)), np.zeros((self.H, self.T))
        to, tl = np.zeros_like(o), np.zeros_like(lse)
        kp, vp, q = f64(self.k), f64(self.v), f64(self.q)
        G = self.H // self.Hkv
        for b, n in enumerate(self.lens):
            a, z = self.cu[b], self.cu[b + 1]
            if a == z:
                continue
            for h in range(self.Hkv):
                k, v = (P.rows(x, self.table[b], n, h, self.page) for x in (kp, vp))
                qh = q[a:z, h * G:(h + 1) * G].transpose(1, 0, 2)
                oh, lh, w = K.attend(qh, k, v, n, scale)
                e = (self.D + 4) * 2.0 ** -23 * ((np.abs(qh) @ np.abs(k).T).max() * abs(scale) if n else 0.0)
                rel = 2.0 ** -8 + 2 * e + 2.0 ** -20 + SUM
                o[a:z, h * G:(h + 1) * G] = oh.transpose(1, 0, 2)
                err = rel * (w @ np.abs(v))
                to[a:z, h * G:(h + 1) * G] = (err + 2.0 ** -8 * (np.abs(oh) + err) + 1e-30).transpose(1, 0, 2)
                lse[h * G:(h + 1) * G, a:z] = lh
                tl[h * G:(h + 1) * G, a:z] = e + SUM + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lh), lh, 0))
        return o, lse, to, tl

    def run(self, cu=True, scale=None, ws=None, **kw):
        return cca.paged_attention(self.q, self.cache, i32(self.table), i32(self.lens), i32(self.cu) if cu else None,
                                   scale=scale, ws=ws, **kw)

    def check(self, cu=True, scale=None, ws=None, rows=None):
        ws = cca.paged_workspace(self.cache, self.q, len(self.lens)) if ws is None else ws
        o, lse = self.run(cu, scale, ws)
        assert cca.attn_status(ws) == 0
        self.compare(o, lse, scale)
        return o, lse

    def compare(self, o, lse, scale=None):
        wo, wl, to, tl = self.want(scale)
        n = self.cu[-1]
        go, gl = f64(o)[:n], f64(lse)[0, :, :n]
        assert np.isfinite(go).all()
        assert (np.abs(go - wo[:n]) <= to[:n]).all(), np.max(np.abs(go - wo[:n]) / to[:n])
        none = np.isneginf(wl[:, :n])
        assert (np.isneginf(gl) == none).all()
        far = np.abs(np.where(none, 0, gl - np.where(none, 0, wl[:, :n])))
        assert (far <= tl[:, :n]).all(), np.max(far / tl[:, :n])


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("lens,nq,H,Hkv,D,page,layout", [
    ([1], [1], 1, 1, 64, 16, "heads"),
    ([100], [1], 4, 1, 128, 16, "heads"),
    ([128], [1], 4, 2, 128, 128, "slots"),
    ([300], [1], 8, 2, 128, 64, "both"),
    ([1000], [1], 32, 8, 128, 64, "heads"),
    ([129, 1, 0, 777], [1, 1, 1, 1], 10, 2, 64, 16, "gaps"),
    ([513], [5], 8, 1, 64, 32, "heads"),
    ([260], [200], 4, 2, 128, 16, "outer"),
    ([700], [700], 3, 3, 128, 256, "slots"),
    ([900, 65, 2000, 31], [400, 65, 1, 0], 10, 2, 128, 64, "heads"),
    ([333, 40], [100, 40], 6, 3, 256, 16, "heads"),
    ([333, 40], [1, 3], 6, 3, 256, 128, "gaps"),
    ([333, 40], [100, 40], 6, 3, 40, 16, "both"),
    ([200, 700], [77, 130], 5, 1, 80, 1024, "slots"),
    ([200, 150], [10, 20], 12, 4, 200, 64, "heads"),
    ([70, 300], [3, 2], 129, 1, 64, 32, "heads"),
    ([64, 200], [2, 70], 512, 2, 64, 16, "slots"),
    ([40], [7], 200, 1, 8, 16, "heads"),
])
def test_attention(lens, nq, H, Hkv, D, page, layout):
    Batch(lens, nq, H, Hkv, D, page, layout, seed=sum(lens) + D).check()


@pytest.mark.parametrize("seed", range(12))
def test_attention_random(seed):
    rng = np.random.default_rng(100 + seed)
    B = int(rng.integers(1, 7))
    Hkv, G = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 4, 5, 8]))
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(3500), B))]
    nq = [int(min(n, np.exp(rng.uniform(0, np.log(600))))) for n in lens]
    Batch(lens, nq, Hkv * G, Hkv, int(rng.choice([8, 24, 64, 72, 96, 128, 136, 192, 256])), int(2 ** rng.integers(4, 11)),
          str(rng.choice(["heads", "slots", "both", "gaps", "outer"])), seed=seed, pad=int(rng.integers(0, 50))).check()


@pytest.mark.parametrize("lens,nq,H,Hkv,D,page", [
    ([900], [700], 32, 32, 64, 64),                     # 192 units: more than there are SMs
    ([5, 1200, 70], [0, 1100, 0], 24, 24, 128, 16),     # among sequences without tokens
    ([2000], [1300], 64, 16, 64, 32),
    ([700], [700], 30, 30, 256, 128),
    ([40], [40], 200, 200, 8, 16),                      # one key tile each
])
def test_one_sequence_of_many_units(lens, nq, H, Hkv, D, page):
    Batch(lens, nq, H, Hkv, D, page, seed=H).check()


def test_queries_that_see_nothing():
    # more new tokens than slots in use: the first ones see none
    b = Batch([3, 0, 200], [10, 4, 250], 4, 2, 64, 16)
    o, lse = b.check()
    assert (f64(o)[:7] == 0).all() and np.isneginf(f64(lse)[0, :, :7]).all()
    assert (f64(o)[10:14] == 0).all() and (f64(o)[14:64] == 0).all()


def test_uniform_tokens_without_offsets():
    b = Batch([50, 300, 129], [3, 3, 3], 8, 2, 128, 32)
    o, lse = b.check(cu=False)
    o2, lse2 = b.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_padding_is_left_alone():
    b = Batch([300, 150], [100, 1], 8, 2, 64, 16, pad=60)
    o, lse = torch.full_like(b.q, 7.0), torch.full((1, 8, b.T), 7.0, device="cuda")
    b.run(o=o, lse=lse)
    b.compare(o, lse)
    assert (o[101:] == 7.0).all() and (lse[..., 101:] == 7.0).all()


@pytest.mark.parametrize("B", [127, 129, 300, 1500])
def test_many_sequences(B):
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 260, B)]
    lens[B // 2] = 5000
    nq = [int(x) for x in rng.integers(0, 3, B)]
    nq[B // 2] = 40
    Batch(lens, nq, 4, 1, 64, 16, seed=B).check()


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.0])
def test_scales(scale):
    Batch([300, 40], [140, 1], 4, 2, 64, 16, seed=5, amp=1.0).check(scale=scale)


def test_strided_queries():
    b = Batch([300, 40], [140, 1], 4, 2, 64, 16, seed=6)
    want_o, want_l = b.run()
    for make in (lambda q: torch.cat((q, q, q), 1)[:, 4:8],                                 # part of a fused projection
                 lambda q: q.transpose(0, 1).contiguous().transpose(0, 1),                  # heads outside tokens
                 lambda q: torch.nn.functional.pad(q, (0, 8))[..., :64]):
        b.q = make(b.q)
        o, lse = b.run()
        assert o.stride() == b.q.stride()
        assert torch.equal(o, want_o) and torch.equal(lse, want_l)


@pytest.mark.parametrize("page,D", [(16, 64), (128, 64), (32, 128), (64, 128), (16, 256), (256, 256)])
def test_values_that_are_not_finite(page, D):
    # NaN and infinity in V reach the rows that see their slot and no other
    b = Batch([700], [300], 4, 2, D, page, seed=7)
    clean_o, clean_l = b.run()
    slots = [(410, 3, math.inf), (450, 60, math.nan), (600, 5, -math.inf), (699, 0, math.nan), (100, 9, math.inf)]
    for j, d, x in slots:
        b.v[b.table[0, j // page], 1, j % page, d] = x
    o, lse = b.run()
    assert torch.equal(lse, clean_l)
    want = f64(clean_o)
    for j, d, x in slots:
        first = max(0, j - 400)
        want[first:, 2:, d] += x
    got = f64(o)
    assert (np.isnan(got) == np.isnan(want)).all() and (np.isposinf(got) == np.isposinf(want)).all()
    assert (np.isneginf(got) == np.isneginf(want)).all()
    fine = np.isfinite(want)
    assert (got[fine] == want[fine]).all()


def test_keys_that_are_not_finite():
    # NaN in K reaches the rows that see its slot and no other
    b = Batch([300], [200], 2, 1, 64, 16, seed=8)
    clean_o, clean_l = b.run()
    b.k[b.table[0, 250 // 16], 0, 250 % 16, 3] = math.nan
    o, lse = b.run()
    assert torch.equal(o[:150], clean_o[:150]) and torch.equal(lse[..., :150], clean_l[..., :150])
    assert o[150:].isnan().all() and lse[..., 150:].isnan().all()


@pytest.mark.parametrize("page", [16, 64])
def test_values_that_are_not_finite_in_every_edge_tile(page):
    # one head to a key/value head: 128 tokens a tile, every one of which hides the ones after it
    b = Batch([400, 130], [390, 130], 2, 2, 128, page, seed=17)
    clean_o, clean_l = b.run()
    for j in (129, 200, 399):
        b.v[b.table[0, j // page], 0, j % page, 7] = math.nan
    o, lse = b.run()
    want = f64(clean_o)
    want[129 - 10:390, 0, 7] = math.nan
    assert np.array_equal(f64(o), want, equal_nan=True) and torch.equal(lse, clean_l)


def test_tables_with_gaps_and_calls_on_other_streams():
    b = Batch([3000, 65, 200], [40, 65, 1], 8, 2, 128, 16, seed=18)
    want = b.run()
    wide = torch.full((3, b.table.shape[1] + 13), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :b.table.shape[1]] = i32(b.table)
    table, lens, cu = wide[:, :b.table.shape[1]], i32(b.lens), i32(b.cu)
    ws = cca.paged_workspace(b.cache, b.q, 3)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        o, lse = cca.paged_attention(b.q, b.cache, table, lens, cu, ws=ws, stream=stream)
        s.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    with torch.cuda.stream(s):
        o, lse = cca.paged_attention(b.q, b.cache, table, lens, cu)
    s.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and cca.attn_status(ws) == 0


def test_shared_pages():
    # two sequences with the same first pages
    b = Batch([96, 130], [3, 5], 4, 2, 64, 16, seed=19)
    b.table[1, :4] = b.table[0, :4]
    b.check()


def test_same_result_every_time():
    b = Batch([3000, 65, 2000, 31], [400, 65, 1, 0], 10, 2, 128, 64)
    ws = cca.paged_workspace(b.cache, b.q, 4)
    o, lse = b.check(ws=ws)
    for _ in range(5):
        o2, lse2 = b.run(ws=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_far_offsets():
    # pages and queries beyond 2^31 elements
    page, Hkv, D = 1024, 8, 128
    pages = (1 << 31) // (page * Hkv * D) + 40
    free = torch.cuda.mem_get_info()[0]
    if free < 14 << 30:
        pytest.skip("needs 14 GiB")
    k, v = (torch.empty((pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rng = np.random.default_rng(9)
    table = np.array([[pages - 1, 0, pages - 7]])
    rows = [bf16(rng, 3 * page, Hkv, D) for _ in range(2)]
    slots = torch.as_tensor(np.concatenate([np.arange(p * page, (p + 1) * page) for p in table[0]]), dtype=torch.int32).cuda()
    cache = cca.PagedCache(k, v)
    cca.paged_store(cache, rows[0], rows[1], slots)
    small = Batch([2500], [30], 16, Hkv, D, page, seed=9)
    for i, p in enumerate(table[0]):
        small.k[small.table[0, i]] = k[p]
        small.v[small.table[0, i]] = v[p]
        assert torch.equal(k[p], rows[0][i * page:(i + 1) * page].transpose(0, 1))
    want = small.run()
    got = cca.paged_attention(small.q, cache, i32(table), i32([2500]), i32([0, 30]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_bad_integers_are_reported():
    b = Batch([300, 40], [20, 1], 4, 2, 64, 16)
    ws = cca.paged_workspace(b.cache, b.q, 2)
    table, lens, cu = i32(b.table), i32(b.lens), i32(b.cu)
    call = lambda t=table, n=lens, c=cu: cca.paged_attention(b.q, b.cache, t, n, c, ws=ws)
    good = call()
    assert cca.attn_status(ws) == 0
    for bad in (1 << 30, -1, b.k.shape[0]):
        t = table.clone()
        t[0, 3] = bad
        o, _ = call(t=t)
        assert cca.attn_status(ws) == 7
        assert torch.equal(o[20:], good[0][20:])
    for n in ([-5, 40], [1 << 30, 40]):
        o, _ = call(n=i32(n))
        assert cca.attn_status(ws) == 7
        assert torch.equal(o[20:], good[0][20:])
    for c in ([0, 1 << 30, 21], [0, 20, 1 << 30], [-4, 20, 21], [0, 20, 5], [21, 0, 21]):
        call(c=i32(c))
        assert cca.attn_status(ws) == 7
    assert torch.equal(call()[0], good[0]) and cca.attn_status(ws) == 0


def test_captured_and_replayed():
    # one graph serves other lengths, other pages and fewer sequences
    b = Batch([700, 130, 64], [1, 1, 1], 8, 2, 128, 16, seed=11)
    c = Batch([20, 900, 400], [1, 0, 2], 8, 2, 128, 16, seed=12, extra=40)
    ws = cca.paged_workspace(b.cache, b.q, 3)
    wide = np.full((3, 60), -1)
    wide[:, :b.table.shape[1]] = b.table
    table, lens, cu = i32(wide), i32(b.lens), i32(b.cu)
    k, v = (torch.zeros((200, 2, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = cca.PagedCache(k, v)
    k[:b.k.shape[0]], v[:b.k.shape[0]] = b.k, b.v
    q = b.q.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, lse = cca.paged_attention(q, cache, table, lens, cu, ws=ws)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = cca.paged_attention(q, cache, table, lens, cu, ws=ws)
    g.replay()
    b.compare(o, lse)
    wide[:] = -1
    wide[:, :c.table.shape[1]] = c.table
    table.copy_(i32(wide))
    lens.copy_(i32(c.lens))
    cu.copy_(i32(c.cu))
    k[:c.k.shape[0]], v[:c.k.shape[0]] = c.k, c.v
    q.copy_(c.q)
    for _ in range(3):
        g.replay()
    c.compare(o, lse)
    assert cca.attn_status(ws) == 0


def test_two_streams_at_once():
    b, c = Batch([3000], [200], 8, 2, 128, 16, seed=13), Batch([9000], [1], 8, 2, 128, 16, seed=14)
    want = b.run(), c.run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for x, s in zip((b, c), streams):
        table, lens, cu = i32(x.table), i32(x.lens), i32(x.cu)
        torch.cuda.synchronize()
        got.append([cca.paged_attention(x.q, x.cache, table, lens, cu, stream=s) for _ in range(10)])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for o, lse in g:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


def test_waits_that_run_out(monkeypatch):
    b = Batch([300, 40], [20, 1], 4, 2, 64, 16)
    ws = cca.paged_workspace(b.cache, b.q, 2)
    good = b.run(ws=ws)
    monkeypatch.setenv("ATTN_TEST_STALL_PRODUCER", "1")
    monkeypatch.setenv("ATTN_WAIT_LIMIT_MS", "50")
    b.run(ws=ws)
    assert cca.attn_status(ws) == 6
    monkeypatch.delenv("ATTN_TEST_STALL_PRODUCER")
    monkeypatch.delenv("ATTN_WAIT_LIMIT_MS")
    o, lse = b.run(ws=ws)
    assert cca.attn_status(ws) == 0 and torch.equal(o, good[0]) and torch.equal(lse, good[1])


# ------------------------------------------------------------------ store

@pytest.mark.parametrize("T,Hkv,D,page,layout", [(1, 1, 8, 16, "heads"), (3, 2, 64, 16, "slots"), (64, 8, 128, 16, "both"),
                                                 (777, 3, 40, 64, "gaps"), (5000, 4, 256, 1024, "outer"),
                                                 (20001, 2, 128, 32, "heads")])
def test_store(T, Hkv, D, page, layout):
    rng = np.random.default_rng(T)
    pages = -(-T // page) + 3
    k, v = pool_of(rng, pages, Hkv, page, D, layout)
    slots = rng.permutation(pages * page)[:T]
    slots[rng.random(T) < 0.2] = -1
    kn, vn = (bf16(rng, T, Hkv, D) for _ in range(2))
    if T == 777:                                                     # parts of a fused projection
        fused = torch.cat((kn, vn), 1)
        kn, vn = fused[:, :Hkv], fused[:, Hkv:]
    want = []
    for pool, rows in ((k, kn), (v, vn)):
        w = f64(pool).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)
        w[slots[slots >= 0]] = f64(rows)[slots >= 0]
        want.append(w.reshape(pages, page, Hkv, D).transpose(0, 2, 1, 3))
    cache = cca.PagedCache(k, v)
    ws = cca.paged_workspace(cache)
    cca.paged_store(cache, kn, vn, i32(slots), ws=ws)
    assert cca.attn_status(ws) == 0
    assert np.array_equal(f64(k), want[0], equal_nan=True) and np.array_equal(f64(v), want[1], equal_nan=True)


def test_store_skips_slots_outside():
    rng = np.random.default_rng(1)
    cache = cca.paged_cache(4, 2, 16, 64)
    ws = cca.paged_workspace(cache)
    rows = bf16(rng, 6, 2, 64)
    cca.paged_store(cache, rows, rows, i32([3, -1, 64, -2, 63, 2 ** 31 - 1]), ws=ws)
    assert cca.attn_status(ws) == 7
    want = torch.zeros_like(cache.k)
    want[0, :, 3], want[3, :, 15] = rows[0], rows[4]
    assert torch.equal(cache.k, want) and torch.equal(cache.v, want)


# ------------------------------------------------------------------ reserve

def random_tables(rng, B, page, most, spare, ld=None):
    lens = rng.integers(0, most * page + 1, B)
    lens[rng.random(B) < 0.2] = 0
    held = -(-lens // page)
    pages = int(held.sum()) + spare
    order = rng.permutation(pages)
    table = np.full((B, most), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = np.full(pages, -1)
    free[:spare] = order[at:]
    return table, lens, free, spare


@pytest.mark.parametrize("B,page,most,spare,T,big,gap", [
    (1, 16, 4, 3, 1, 1, 0), (2, 16, 4, 8, 40, 17, 3), (7, 32, 5, 4, 100, 9, 0), (64, 16, 40, 60, 64, 1, 0),
    (300, 64, 6, 150, 9000, 40, 5), (1024, 16, 9, 900, 4096, 4, 0), (1025, 16, 9, 900, 4097, 4, 0),
    (5000, 128, 3, 4000, 40000, 7, 1), (3, 1024, 20, 30, 50000, 12000, 0), (2500, 16, 4, 100, 3000, 1, 0)])
@pytest.mark.parametrize("seed", [0, 1])
def test_reserve(B, page, most, spare, T, big, gap, seed):
    rng = np.random.default_rng(1000 * seed + B)
    table, lens, free, n_free = random_tables(rng, B, page, most, spare)
    add = rng.integers(0, big + 1, B)
    add[rng.random(B) < 0.15] = -1
    wt, wl, wf, wn, wcu, ws_, refused = P.reserve(table, lens, free, n_free, add, page, T)
    assert wcu[-1] <= T
    wide = torch.full((B, most + gap), 12345, dtype=torch.int32, device="cuda")
    wide[:, :most] = i32(table)
    tables = cca.PagedTables(wide[:, :most], i32(lens), i32(free), i32([n_free]), page)
    ws = cca.paged_workspace(tables=tables)
    out, n_out = torch.full_like(tables.lens, 5), torch.full_like(tables.n_free, 5)
    for again in range(2):                           # apart from what it reads, then in place
        given = dict(lens_out=out, n_free_out=n_out) if again == 0 else {}
        cu, slots = cca.paged_reserve(tables, i32(add), T, ws=ws, **given)
        assert cca.attn_status(ws) == (8 if refused else 0)
        got_l, got_n = (out, n_out) if again == 0 else (tables.lens, tables.n_free)
        assert np.array_equal(cu.cpu().numpy(), wcu) and np.array_equal(slots.cpu().numpy(), ws_)
        assert np.array_equal(got_l.cpu().numpy(), wl) and int(got_n) == wn
        assert np.array_equal(tables.table.cpu().numpy(), wt) and np.array_equal(tables.free.cpu().numpy(), wf)
        assert (wide[:, most:] == 12345).all()


def test_reserve_reports_bad_integers():
    page, most = 16, 4
    make = lambda lens=(10, 20), free=(2, 3, 4), n=(3,): cca.PagedTables(
        i32([[0, -1, -1, -1], [1, 5, -1, -1]]), i32(lens), i32(free), i32(n), page)
    ws = cca.paged_workspace(tables=make())
    t = make(lens=(10, 1000))
    _, slots = cca.paged_reserve(t, i32([1, 0]), 4, ws=ws)
    assert cca.attn_status(ws) == 7 and slots.tolist() == [10, -1, -1, -1] and t.lens.tolist() == [11, 64]
    t = make(n=(99,))                                # more on the stack than it holds
    cca.paged_reserve(t, i32([10, 0]), 10, ws=ws)
    assert cca.attn_status(ws) == 7 and t.table[0, 1] == 4 and int(t.n_free) == 2
    t = make(free=(2, 3, 4000))                      # a free page that is none
    _, slots = cca.paged_reserve(t, i32([10, 0]), 10, ws=ws)
    assert cca.attn_status(ws) == 7 and slots.tolist() == [10, 11, 12, 13, 14, 15, -1, -1, -1, -1]
    t = make()                                       # pages put back beyond the stack
    cca.paged_reserve(t, i32([-1, -1]), 4, ws=ws)
    assert cca.attn_status(ws) == 7 and int(t.n_free) == 3 and t.free.tolist() == [2, 3, 4]
    t = make()                                       # more tokens than slots were asked for
    cu, slots = cca.paged_reserve(t, i32([3, 4]), 5, ws=ws)
    assert cca.attn_status(ws) == 7 and cu.tolist() == [0, 3, 5] and slots.tolist() == [10, 11, 12, -1, -1]
    assert t.lens.tolist() == [13, 20]
    t = make()                                       # huge wishes
    cu, slots = cca.paged_reserve(t, i32([2 ** 31 - 1, 2 ** 31 - 1]), 5, ws=ws)
    assert cca.attn_status(ws) == 7 and cu.tolist() == [0, 5, 5] and slots.tolist() == [-1] * 5 and int(t.n_free) == 3


def test_reserve_and_store_on_another_stream():
    rng = np.random.default_rng(30)
    k, v = bf16(rng, 50, 2, 64), bf16(rng, 50, 2, 64)
    add = i32([30, 20])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = None
    for stream in (None, s, s.cuda_stream):
        cache, tables = cca.paged_cache(9, 2, 16, 64), cca.paged_tables(2, 4, 9, 16)
        torch.cuda.synchronize()
        for _ in range(2):                           # 60 slots of one sequence, 40 of the other, by calls that allocate
            cu, slots = cca.paged_reserve(tables, add, 50, stream=stream)
            cca.paged_store(cache, k, v, slots, stream=stream)
        torch.cuda.synchronize()
        got = [x.clone() for x in (cache.k, cache.v, tables.table, tables.lens, tables.n_free, cu, slots)]
        assert want is None or all(torch.equal(a, b) for a, b in zip(got, want))
        want = got
    assert tables.lens.tolist() == [60, 40] and tables.n_free.tolist() == [2]
    assert tables.table.tolist() == [[0, 1, 4, 5], [2, 3, 6, -1]]


# ------------------------------------------------------------------ a run of them together

@pytest.mark.parametrize("graph", [False, True])
def test_serving_steps(graph):
    """Prompts in chunks, decoding, ends and new prompts, against the dense forward of each sequence."""
    rng = np.random.default_rng(21)
    B, H, Hkv, D, page, pages, most, T = 4, 8, 2, 128, 16, 80, 40, 160
    cache, tables = cca.paged_cache(pages, Hkv, page, D), cca.paged_tables(B, most, pages, page)
    q, k, v = (torch.zeros((T, n, D), dtype=torch.bfloat16, device="cuda") for n in (H, Hkv, Hkv))
    add = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = cca.paged_workspace(cache, q, B, tables)

    def step():
        cu, slots = cca.paged_reserve(tables, add, T, ws=ws)
        cca.paged_store(cache, k, v, slots, ws=ws)
        return cca.paged_attention(q, cache, tables.table, tables.lens, cu, ws=ws)

    if graph:
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse = step()
    plans = [[100, 30, 0, 20], [1, 60, 140 - 61, 1], [1, 1, 1, 1], [-1, 1, 60, 1], [90, 1, -1, 1], [1, 1, 50, 1], [1, 1, 1, 1]]
    seen = [[] for _ in range(B)]                    # rows of each sequence so far
    for plan in plans:
        n = sum(max(x, 0) for x in plan)
        for t in (q, k, v):
            t.copy_(bf16(rng, *t.shape))
        add.copy_(i32(plan))
        if graph:
            g.replay()
        else:
            o, lse = step()
        at = 0
        for b, x in enumerate(plan):
            if x < 0:
                seen[b] = []
                continue
            if x == 0:
                continue
            seen[b].append((q[at:at + x].clone(), k[at:at + x].clone(), v[at:at + x].clone()))
            qs, ks, vs = (torch.cat(z) for z in zip(*seen[b]))
            L = qs.shape[0]
            wo, wl = cca.forward(qs, ks, vs, [(0, L, 0, 0)], packed=True)
            # two roundings of O and of each weight apart, and partial sums in another order
            tol = (4 * 2.0 ** -8 + 2 * SUM) * float(vs.abs().max())
            assert (o[at:at + x].float() - wo[L - x:].float()).abs().max() <= tol
            assert (lse[0, :, at:at + x] - wl[0, :, L - x:]).abs().max() <= 2 * SUM + 2.0 ** -16
            at += x
    assert cca.attn_status(ws) == 0
    held = sum(-(-sum(r[0].shape[0] for r in s) // page) for s in seen)
    assert int(tables.n_free) == pages - held
