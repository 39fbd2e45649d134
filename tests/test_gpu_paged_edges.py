"""The paged cache's calls at their edges: offsets out of order, calls as their documents allow them.
Outputs are compared with those of a call that has to make the same ones, bit for bit."""
import math

import numpy as np
import pytest
import torch

import chunked_causal_attention_gb300 as cca
from test_gpu_paged import Batch, bf16, built, i32      # noqa: F401 (built: the fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ offsets that leave [0, T] or descend

def nearest(cu, T):
    """Each offset the nearest one in [the one before it, T]."""
    return np.maximum.accumulate(np.clip(np.asarray(cu, dtype=np.int64), 0, T))


def check_offsets(b, cu):
    """Rows of a call with these offsets are those of a call with the nearest ones, the others are left alone."""
    ws = cca.paged_workspace(b.cache, b.q, len(b.lens))
    good = nearest(cu, b.T)
    outs = []
    for x, status in ((good, 0), (cu, 7)):
        o, lse = torch.full_like(b.q, 7.0), torch.full((1, b.H, b.T), 7.0, device="cuda")
        cca.paged_attention(b.q, b.cache, i32(b.table), i32(b.lens), i32(x), o=o, lse=lse, ws=ws)
        assert cca.attn_status(ws) == status
        outs.append((o, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    for o, lse in outs:
        for rows in (slice(0, good[0]), slice(good[-1], b.T)):
            assert (o[rows] == 7.0).all() and (lse[..., rows] == 7.0).all()
        assert not (o[good[0]:good[-1]] == 7.0).all(-1).any()


@pytest.mark.parametrize("cu", [[-4, 20, 21], [0, 20, 1 << 30], [-2 ** 31, 20, 2 ** 31 - 1], [0, -1, 21]])
def test_offsets_outside(cu):
    check_offsets(Batch([300, 40], [20, 1], 4, 2, 64, 16), cu)


@pytest.mark.parametrize("cu", [[0, 20, 5], [21, 0, 21], [9, 3, 2]])
def test_offsets_that_descend(cu):
    check_offsets(Batch([300, 40], [20, 1], 4, 2, 64, 16), cu)


@pytest.mark.parametrize("cu", [[0, 50, 20, 22, 30], [10, 0, 60, 30, 1000], [-5, 30, 30, 10, 40], [60, 61, 5, 9, 61]])
@pytest.mark.parametrize("page", [16, 128])
def test_offsets_that_descend_past_others(cu, page):
    check_offsets(Batch([2000, 129, 700, 64], [50, 1, 5, 4], 8, 2, 128, page, seed=40), cu)


@pytest.mark.parametrize("B", [40, 1200, 3000])
def test_offsets_at_random(B):
    # more sequences than a warp has lanes, and more in a lane's run
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(1, 200, B)]
    lens[B // 3] = 4000
    b = Batch(lens, [1] * B, 4, 2, 64, 16, seed=B, pad=37)
    cu = b.cu.copy()
    at = rng.choice(B + 1, 6, replace=False)
    cu[at] = rng.integers(-50, b.T + 50, 6)
    cu[0] = -3
    check_offsets(b, cu)
    check_offsets(b, np.concatenate([[-2 ** 31], rng.integers(-2 ** 31, 2 ** 31 - 1, B)]))
    check_offsets(b, np.sort(rng.integers(-40, b.T + 40, B + 1))[::-1].copy())


# ------------------------------------------------------------------ many sequences

def test_tens_of_thousands_of_sequences():
    # runs of hundreds of sequences a lane: every block goes on in a run where it found its item before
    B = 20000
    rng = np.random.default_rng(50)
    lens = [int(x) for x in rng.integers(0, 30, B)]
    nq = [int(x) for x in rng.integers(0, 2, B)]
    for b, n, q in ((3, 3000, 9), (B // 2, 9000, 200), (B - 1, 700, 1)):
        lens[b], nq[b] = n, q
    Batch(lens, nq, 2, 1, 64, 16, seed=50).check()


# ------------------------------------------------------------------ the calls with every array given

def test_calls_with_every_array_given():
    """attn_paged_reserve, attn_paged_store and attn_paged_attend do what the handles' calls do."""
    rng = np.random.default_rng(60)
    B, H, Hkv, D, page, pages, most, T = 3, 8, 2, 64, 16, 40, 20, 120
    q, k, v = (bf16(rng, T, n, D) for n in (H, Hkv, Hkv))
    cache, tables = cca.paged_cache(pages, Hkv, page, D), cca.paged_tables(B, most, pages, page)
    other, t = cca.paged_cache(pages, Hkv, page, D), cca.paged_tables(B, most, pages, page)
    ws = cca.paged_workspace(cache, q, B, tables)
    shape, rows = cca.shape_of(q, None, True), cca.shape_of(k, 1.0, True)
    for plan in ([70, 0, 45], [1, 30, -1], [1, 1, 90]):
        add = i32(plan)
        cu, slots = cca.paged_reserve(tables, add, T, ws=ws)
        cca.paged_store(cache, k, v, slots, ws=ws)
        want = cca.paged_attention(q, cache, tables.table, tables.lens, cu, ws=ws)
        cu2, slots2 = torch.empty_like(cu), torch.empty_like(slots)
        o, lse = torch.empty_like(q), torch.empty((1, H, T), device="cuda")
        cca.attn_paged_reserve(add, t.lens, page, t.n_free, t.free, t.table, t.lens, t.n_free, cu2, slots2, ws)
        cca.attn_paged_store(k, v, rows, other.desc, slots2, ws)
        cca.attn_paged_attend(q, shape, other.desc, t.table, t.lens, cu2, o, lse, ws)
        assert cca.attn_status(ws) == 0
        n = sum(max(x, 0) for x in plan)
        for a, b in ((cu, cu2), (slots, slots2), (tables.table, t.table), (tables.lens, t.lens), (tables.free, t.free),
                     (tables.n_free, t.n_free), (cache.k, other.k), (cache.v, other.v), (want[0][:n], o[:n]),
                     (want[1][..., :n], lse[..., :n])):
            assert torch.equal(a, b)
    # T / B tokens of each without offsets
    cca.attn_paged_attend(q, shape, other.desc, t.table, t.lens, None, o, lse, ws)
    want = cca.paged_attention(q, cache, tables.table, tables.lens, ws=ws)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and cca.attn_status(ws) == 0
    # what they refuse before the library is called
    for call in (lambda: cca.attn_paged_reserve(add, t.lens[:2], page, t.n_free, t.free, t.table, t.lens, t.n_free, cu2, slots2, ws),
                 lambda: cca.attn_paged_reserve(add.cpu(), t.lens, page, t.n_free, t.free, t.table, t.lens, t.n_free, cu2, slots2, ws),
                 lambda: cca.attn_paged_reserve(add, t.lens, page, t.n_free, t.free, t.table.T, t.lens, t.n_free, cu2, slots2, ws),
                 lambda: cca.attn_paged_store(k, v[:, :, ::2], rows, other.desc, slots2, ws),
                 lambda: cca.attn_paged_store(k, v, rows, other.desc, slots2[1:], ws),
                 lambda: cca.attn_paged_attend(q, shape, other.desc, t.table, t.lens, cu2, o.float(), lse, ws),
                 lambda: cca.attn_paged_attend(q, shape, other.desc, t.table, t.lens, cu2[1:], o, lse, ws),
                 lambda: cca.attn_paged_attend(q, shape, other.desc, t.table.long(), t.lens, cu2, o, lse, ws)):
        with pytest.raises(cca.AttnError) as e:
            call()
        assert e.value.status == 1


# ------------------------------------------------------------------ pages of several sequences

def test_a_shared_page_is_copied_before_it_is_written():
    """Two sequences begin with the same pages; the second one's last page, half full, is stored in a page of its own
    before both go on. Rows of the pool are the call's rows, and no slot is both read and written."""
    page, Hkv, D = 16, 2, 64
    b = Batch([40, 40], [1, 1], 4, Hkv, D, page, seed=61, extra=3)
    b.table[1, :2] = b.table[0, :2]                  # two full pages of both, eight slots of the third
    own = int(b.table[1, 2])
    for pool in (b.k, b.v):
        pool[own] = math.nan
    at = int(b.table[0, 2])
    rows = [pool[at].transpose(0, 1) for pool in (b.k, b.v)]      # [page, Hkv, D], views of the pool
    slots = [own * page + i if i < 8 else -1 for i in range(page)]
    ws = cca.paged_workspace(b.cache, b.q, 2)
    cca.paged_store(b.cache, *rows, i32(slots), ws=ws)
    new = [bf16(np.random.default_rng(62 + i), 2, Hkv, D) for i in range(2)]
    cca.paged_store(b.cache, *new, i32([at * page + 8, own * page + 8]), ws=ws)
    assert cca.attn_status(ws) == 0
    for pool, n in zip((b.k, b.v), new):
        assert torch.equal(pool[own, :, :8], pool[at, :, :8])
        assert torch.equal(pool[at, :, 8], n[0]) and torch.equal(pool[own, :, 8], n[1])
    b.lens = [41, 41]
    b.check()
