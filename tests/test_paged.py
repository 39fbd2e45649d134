"""The paged cache without a GPU: argument checks of its entry points (on the host,
before any CUDA call) and hand-worked reservations of the oracle."""
import ctypes
import os

import numpy as np
import pytest
import torch

import chunked_causal_attention_gb300 as cca
from chunked_causal_attention_gb300 import _lib
from oracle import paged as P

FAKE, WS = ctypes.c_void_p(4096), ctypes.c_void_p(1 << 20)
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(_lib.LIB_PATH):
        from chunked_causal_attention_gb300 import build
        build.build()


def cache(pages=9, Hkv=2, page=16, D=64, sp=None, sh=None, st=None, k=1 << 24, v=2 << 24):
    st = D if st is None else st
    sh = page * st if sh is None else sh
    return _lib.attn_paged_cache(pages, Hkv, page, D, Hkv * sh if sp is None else sp, sh, st, k, v)


def shape(T=6, H=4, D=64, B=1, scale=0.125):
    return cca.make_shape(B, H, T, D, T * H * D, H * D, D, scale)


def attend(s=None, c=None, q=FAKE, table=FAKE, ld=8, most=8, lens=FAKE, cu=FAKE, B=2, o=ctypes.c_void_p(1 << 30), lse=FAKE,
           ws=WS, n=BIG):
    s, c = s or shape(), c or cache()
    return cca.lib().attn_paged_attend(q, ctypes.byref(s), ctypes.byref(c), table, ld, most, lens, cu, B, o, lse, ws, n, None)


def store(s=None, c=None, k=FAKE, v=FAKE, slots=FAKE, ws=WS, n=BIG):
    s, c = s or shape(H=2), c or cache()
    return cca.lib().attn_paged_store(k, v, ctypes.byref(s), ctypes.byref(c), slots, ws, n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(pages=0), 1), (dict(pages=1 << 27), 1), (dict(Hkv=0), 1), (dict(page=8), 1), (dict(page=48), 1), (dict(page=2048), 1),
    (dict(page=0), 1), (dict(page=-16), 1), (dict(D=0), 1), (dict(D=12), 3), (dict(D=264), 3),
    (dict(st=68), 2), (dict(sp=4100), 2), (dict(sh=0), 1), (dict(st=-64), 1), (dict(st=56), 1), (dict(sh=512), 1), (dict(sp=1024), 1),
    (dict(k=0), 1), (dict(v=0), 1), (dict(k=(1 << 24) + 8), 2)])
def test_cache_checks(bad, status):
    n = ctypes.c_size_t(0)
    c = cache(**bad)
    launches = cca.kernel_launches()
    L = cca.lib()
    assert L.attn_paged_workspace_size(ctypes.byref(c), None, 1, _lib.PAGED_STORE, ctypes.byref(n)) == status
    assert attend(c=c) == status and store(c=c) == status
    assert cca.kernel_launches() == launches


def test_workspace_sizes():
    c = cache()
    assert cca.attn_paged_workspace_size(c, None, 1, cca.PAGED_STORE) == 256
    assert cca.attn_paged_workspace_size(None, None, 5, cca.PAGED_RESERVE) >= 256 + 5 * 20
    one = cca.attn_paged_workspace_size(c, shape(T=1), 1, cca.PAGED_ATTEND)
    assert 256 < one <= cca.attn_paged_workspace_size(c, shape(T=500), 7, cca.PAGED_ATTEND)
    for c_, s, B, op in ((c, None, 1, cca.PAGED_ATTEND), (None, shape(), 1, cca.PAGED_ATTEND), (c, shape(), 0, cca.PAGED_ATTEND),
                         (None, None, 0, cca.PAGED_RESERVE), (c, shape(), 1, 3), (c, shape(), 1, -1),
                         (c, shape(H=3), 1, cca.PAGED_ATTEND), (c, shape(D=128), 1, cca.PAGED_ATTEND),
                         (c, shape(B=2), 1, cca.PAGED_ATTEND)):
        with pytest.raises(cca.AttnError) as e:
            cca.attn_paged_workspace_size(c_, s, B, op)
        assert e.value.status == 1


def test_attend_refuses():
    launches = cca.kernel_launches()
    for arg in ("q", "table", "lens", "o", "lse"):
        assert attend(**{arg: None}) == 1
    assert attend(q=ctypes.c_void_p(4104)) == 2 and attend(lse=ctypes.c_void_p(4104)) == 2
    assert attend(lens=ctypes.c_void_p(4098)) == 2 and attend(cu=ctypes.c_void_p(4098)) == 2
    assert attend(ws=None) == 4 and attend(n=256) == 4 and attend(ws=ctypes.c_void_p(4096 + 64)) == 2
    assert attend(B=0) == 1 and attend(ld=7) == 1 and attend(most=0) == 1 and attend(most=1 << 27, ld=1 << 27) == 1
    assert attend(cu=None, B=4) == 1                                            # 6 tokens of 4 sequences
    assert attend(o=FAKE) == 1 and attend(o=ctypes.c_void_p(4096 + 512)) == 1  # the queries' memory
    assert attend(s=shape(H=3)) == 1 and attend(s=shape(D=128)) == 1 and attend(s=shape(B=2)) == 1
    assert attend(s=cca.make_shape(1, 4, 6, 64, 1536, 128, 64, 0.1)) == 1      # rows that overlap
    assert attend(s=cca.make_shape(1, 4, 6, 64, 1536, 260, 64, 0.1)) == 2
    assert attend(s=shape(scale=float("inf"))) == 1
    assert attend(s=shape(T=1 << 29, H=8)) == 1                                 # 2^32 rows
    assert cca.kernel_launches() == launches


def test_store_refuses():
    launches = cca.kernel_launches()
    for arg in ("k", "v", "slots"):
        assert store(**{arg: None}) == 1
    assert store(k=ctypes.c_void_p(4104)) == 2 and store(slots=ctypes.c_void_p(4098)) == 2
    assert store(ws=None) == 4 and store(n=255) == 4 and store(ws=ctypes.c_void_p(4096 + 64)) == 2
    assert store(s=shape(H=4)) == 1 and store(s=shape(H=2, D=128)) == 1 and store(s=shape(H=2, B=2)) == 1
    assert store(s=shape(T=1 << 28, H=2)) == 1                                  # 2^32 pieces
    assert cca.kernel_launches() == launches


def test_reserve_refuses():
    launches = cca.kernel_launches()
    names = ("add", "lens", "n_free", "free", "table", "lens_out", "n_free_out", "cu", "slots")
    at = {n: (i + 1) << 24 for i, n in enumerate(names)}

    def call(B=3, page=16, pages=40, ld=8, most=8, T=10, ws=WS, n=BIG, **ptrs):
        p = {k: ctypes.c_void_p(v) if v else None for k, v in {**at, **ptrs}.items()}
        return cca.lib().attn_paged_reserve(p["add"], p["lens"], B, page, pages, p["n_free"], p["free"], p["table"], ld, most,
                                            p["lens_out"], p["n_free_out"], p["cu"], p["slots"], T, ws, n, None)

    for name in names:
        assert call(**{name: 0}) == 1
        assert call(**{name: at[name] + 2}) == 2
    for bad in (dict(B=0), dict(page=8), dict(page=24), dict(pages=0), dict(pages=1 << 27), dict(ld=7), dict(most=0), dict(T=0),
                dict(T=1 << 30), dict(B=1 << 31), dict(most=1 << 27, ld=1 << 27)):
        assert call(**bad) == 1, bad
    assert call(ws=None) == 4 and call(n=300) == 4 and call(ws=ctypes.c_void_p(4096 + 64)) == 2
    # what is written overlaps something else
    assert call(slots=at["add"]) == 1 and call(cu=at["lens"]) == 1 and call(lens_out=at["lens"] + 4) == 1
    assert call(table=at["free"]) == 1 and call(n_free_out=at["free"]) == 1 and call(lens_out=at["add"]) == 1
    assert call(n_free_out=at["lens"]) == 1 and call(lens_out=at["lens"], slots=at["lens"]) == 1
    one = dict(B=1, T=1, ld=1, most=1, pages=1)             # arrays of the same size
    for name in names[3:]:
        for other in names:
            if name != other and (name, other) not in (("lens_out", "lens"), ("n_free_out", "n_free")):
                assert call(**one, **{name: at[other]}) == 1, (name, other)
    assert cca.kernel_launches() == launches


def test_python_refuses():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    for k, v in ((bf(4, 2, 16, 64), bf(4, 2, 16, 32)), (bf(4, 2, 16, 64), bf(4, 16, 2, 64).transpose(1, 2)),
                 (torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 16, 64)), (bf(2, 16, 64), bf(2, 16, 64)),
                 (bf(4, 2, 24, 64), bf(4, 2, 24, 64)), (bf(4, 2, 64, 16).transpose(2, 3), bf(4, 2, 64, 16).transpose(2, 3))):
        with pytest.raises(cca.AttnError):
            cca.PagedCache(k, v)
    ok = dict(table=i32(2, 4), lens=i32(2), free=i32(8), n_free=i32(1), page=16)
    cca.PagedTables(**ok)
    for bad in (dict(table=i32(8)), dict(table=i32(4, 2).T), dict(lens=i32(3)), dict(free=i32(8).long()), dict(n_free=i32(2)),
                dict(page=24), dict(page=2048), dict(lens=i32(4)[::2])):
        with pytest.raises(cca.AttnError):
            cca.PagedTables(**{**ok, **bad})
    # tensors that are not on a GPU, of another type or size
    c, t = cca.paged_cache(4, 2, 16, 64, device="cpu"), cca.paged_tables(2, 4, 4, 16, device="cpu")
    ws = cca.paged_workspace(c, bf(3, 4, 64), 2, t)
    for call in (lambda: cca.paged_store(c, bf(3, 2, 64), bf(3, 2, 64), i32(3), ws=ws),
                 lambda: cca.paged_attention(bf(3, 4, 64), c, t.table, t.lens, i32(3), ws=ws),
                 lambda: cca.paged_reserve(t, i32(2), 3, ws=ws),
                 lambda: cca.paged_attention(bf(3, 4, 32), c, t.table, t.lens, i32(3), ws=ws)):
        with pytest.raises(cca.AttnError) as e:
            call()
        assert e.value.status == 1


def test_new_tables_are_empty():
    t = cca.paged_tables(3, 5, 7, 32, device="cpu")
    assert t.table.shape == (3, 5) and t.lens.tolist() == [0, 0, 0] and t.n_free.tolist() == [7]
    assert t.free.tolist() == [6, 5, 4, 3, 2, 1, 0]                            # page 0 is taken first


def test_oracle_reserve_by_hand():
    # pages of 16; stack 7 8 9 (9 on top); b0 grows over a page's end, b1 ends, b2 begins, b3 finds no page,
    # b4 needs none, b5 would find one but comes after b3
    table = np.full((6, 3), -1)
    table[0, 0], table[1, :2], table[3, 0], table[4, 0], table[5, 0] = 3, (4, 5), 6, 2, 1
    lens, add = [15, 20, 0, 16, 1, 16], [2, -1, 33, 20, 5, 1]
    t, n, free, left, cu, slots, refused = P.reserve(table, lens, [7, 8, 9, -1, -1, -1], 3, add, 16, 63)
    # 4 and 5 go on top of 9: b0 takes 5; b2 takes 4, 9, 8; b3 needs two more and one (7) is left
    assert t[0].tolist() == [3, 5, -1] and t[2].tolist() == [4, 9, 8]
    assert n.tolist() == [17, 0, 33, 16, 6, 16] and refused == [3, 5] and left == 1
    assert free.tolist() == [7, 8, 9, 4, 5, -1]
    assert cu.tolist() == [0, 2, 2, 35, 55, 60, 61]
    assert slots[:2].tolist() == [3 * 16 + 15, 5 * 16]
    assert slots[2:35].tolist() == [64 + i for i in range(16)] + [144 + i for i in range(16)] + [128]
    assert (slots[35:55] == -1).all() and slots[55:60].tolist() == [33, 34, 35, 36, 37] and (slots[60:] == -1).all()


def test_oracle_reserve_table_full():
    t, n, _, left, _, slots, refused = P.reserve(np.array([[0, -1], [1, -1]]), [10, 16], [2, 3], 2, [30, 1], 16, 31)
    assert refused == [0] and n.tolist() == [10, 17] and t.tolist() == [[0, -1], [1, 3]] and left == 1
    assert slots.tolist() == [-1] * 30 + [48]


def test_oracle_rows():
    pool = np.arange(4 * 1 * 2 * 1).reshape(4, 1, 2, 1)
    assert P.rows(pool, [3, 0, 2], 3, 0, 2)[:, 0].tolist() == [6, 7, 0]


def test_most_sequences():
    most = 1 << 20
    assert cca.attn_paged_workspace_size(None, None, most, cca.PAGED_RESERVE) >= 20 * most
    for op, args in ((cca.PAGED_RESERVE, (None, None)), (cca.PAGED_ATTEND, (cache(), shape()))):
        with pytest.raises(cca.AttnError) as e:
            cca.attn_paged_workspace_size(*args, most + 1, op)
        assert e.value.status == 1


def test_scale_of_a_tensor_is_read_every_time():
    c, q, scale = cca.paged_cache(4, 2, 16, 64, device="cpu"), torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.tensor(0.5)
    assert c._shape(q, scale)._obj.scale == 0.5
    scale.fill_(0.25)
    assert c._shape(q, scale)._obj.scale == 0.25
    assert c._shape(q, np.array(2.0))._obj.scale == 2.0 and c._shape(q, None)._obj.scale == 0.125
