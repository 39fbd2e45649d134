"""The 4-bit cache's and the key mass's entry points without a GPU: sizes and
arguments are checked on the host, before any CUDA call."""
import ctypes
import os

import pytest
import torch

import chunked_causal_attention_gb300 as cca
from chunked_causal_attention_gb300 import _lib

FAKE, WS = ctypes.c_void_p(4096), ctypes.c_void_p(1 << 20)
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(_lib.LIB_PATH):
        from chunked_causal_attention_gb300 import build
        build.build()


def cache(B=2, Hkv=2, cap=64, D=64, sb=None, sh=None, ptrs=None, ks=1.0, vs=1.0):
    sh = cap if sh is None else sh
    sb = Hkv * sh if sb is None else sb
    return _lib.attn_kv4_cache(B, Hkv, cap, D, sb, sh, *(ptrs or (1 << 24, 2 << 24, 3 << 24, 4 << 24)), ks, vs)


def shape(B=2, H=4, T=1, D=64):
    return cca.make_shape(B, H, T, D, H * T * D, D, T * D, 0.125)


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), 1), (dict(Hkv=0), 1), (dict(cap=0), 1), (dict(cap=-16), 1), (dict(D=0), 1), (dict(cap=1 << 31), 1),
    (dict(D=12), 3), (dict(D=264), 3), (dict(D=4), 3),
    (dict(cap=60), 2), (dict(sh=72, sb=160), 2), (dict(sb=136), 2), (dict(sh=48), 1), (dict(sb=48), 1), (dict(sb=0), 1),
    (dict(ks=0.3), 1), (dict(vs=0.0), 1), (dict(ks=-1.0), 1), (dict(vs=float("inf")), 1), (dict(ks=float("nan")), 1),
    (dict(ks=2.0 ** 65), 1), (dict(vs=2.0 ** -65), 1),
    (dict(ptrs=(0, 2 << 24, 3 << 24, 4 << 24)), 1), (dict(ptrs=(8, 2 << 24, 3 << 24, 4 << 24)), 2)])
def test_cache_checks(bad, status):
    n = ctypes.c_size_t(0)
    c = cache(**bad)
    launches = cca.kernel_launches()
    L = cca.lib()
    assert L.attn_kv4_workspace_size(ctypes.byref(c), None, 0, ctypes.byref(n)) == status
    s = shape()
    assert L.attn_kv4_attend(FAKE, ctypes.byref(s), ctypes.byref(c), FAKE, FAKE, FAKE, None, None, 0, WS, BIG, None) == status
    assert cca.kernel_launches() == launches


def test_workspace_sizes():
    c = cache()
    assert cca.attn_kv4_workspace_size(c, None, cca.KV4_ROWS) == 256
    plain = cca.attn_kv4_workspace_size(c, shape(), cca.KV4_ATTEND)
    assert 256 <= plain <= cca.attn_kv4_workspace_size(c, shape(), cca.KV4_ATTEND_MASS)
    for op, s in ((3, shape()), (-1, shape()), (cca.KV4_ATTEND, None)):
        with pytest.raises(cca.AttnError) as e:
            cca.attn_kv4_workspace_size(c, s, op)
        assert e.value.status == 1
    for bad in (shape(D=128), shape(B=1), shape(H=3)):
        with pytest.raises(cca.AttnError) as e:
            cca.attn_kv4_workspace_size(c, bad, cca.KV4_ATTEND)
        assert e.value.status == 1
    for ts in (2.0 ** -64, 2.0 ** 64, 1.0, 0.5):
        assert cca.attn_kv4_workspace_size(cache(ks=ts, vs=ts), None, cca.KV4_ROWS) == 256


def test_rows_calls_refuse():
    L = cca.lib()
    launches = cca.kernel_launches()

    def call(s=None, c=None, k=FAKE, v=FAKE, pos=FAKE, cu=None, ws=WS, n=BIG, load=False):
        s = s or cca.make_shape(2, 2, 5, 64, 640, 64, 320, 1.0)
        c = c or cache()
        if load:
            return L.attn_kv4_load(ctypes.byref(c), pos, cu, ctypes.byref(s), k, v, ws, n, None)
        return L.attn_kv4_store(k, v, ctypes.byref(s), ctypes.byref(c), pos, cu, ws, n, None)

    for load in (False, True):
        for arg in ("k", "v", "pos"):
            assert call(load=load, **{arg: None}) == 1
        assert call(load=load, k=ctypes.c_void_p(4104)) == 2
        assert call(load=load, pos=ctypes.c_void_p(4098)) == 2
        assert call(load=load, ws=None) == 4 and call(load=load, n=255) == 4
        assert call(load=load, ws=ctypes.c_void_p(4096 + 64)) == 2
        assert call(load=load, s=cca.make_shape(1, 2, 5, 64, 640, 64, 320, 1.0)) == 1          # B differs, not packed
        assert call(load=load, cu=FAKE) == 1                                                      # packed has B = 1
        assert call(load=load, s=cca.make_shape(2, 4, 5, 64, 1280, 64, 320, 1.0)) == 1         # heads differ
        assert call(load=load, s=cca.make_shape(2, 2, 5, 128, 1280, 128, 640, 1.0)) == 1       # D differs
        big = cca.make_shape(1, 2, 1 << 30, 64, 1 << 38, 128, 64, 1.0)
        assert call(load=load, s=big, cu=FAKE) == 1                                               # 2^31 rows
    assert cca.kernel_launches() == launches


def test_attend_refuses():
    L = cca.lib()
    launches = cca.kernel_launches()

    def call(s=None, c=None, q=FAKE, lens=FAKE, o=FAKE, lse=FAKE, mi=None, mo=None, ld=0, ws=WS, n=BIG):
        s, c = s or shape(), c or cache()
        return L.attn_kv4_attend(q, ctypes.byref(s), ctypes.byref(c), lens, o, lse, mi, mo, ld, ws, n, None)

    for arg in ("q", "lens", "o", "lse"):
        assert call(**{arg: None}) == 1
    assert call(q=ctypes.c_void_p(4104)) == 2 and call(lse=ctypes.c_void_p(4104)) == 2
    assert call(ws=None) == 4 and call(n=0) == 4
    assert call(s=shape(H=3)) == 1 and call(s=shape(D=128)) == 1 and call(s=shape(B=3)) == 1
    assert call(s=cca.make_shape(2, 4, 1, 64, 256, 60, 64, 0.1)) == 2
    assert call(s=cca.make_shape(2, 4, 1, 64, 256, 64, 64, float("nan"))) == 1
    assert call(mi=FAKE) == 1                                                   # weights to add, nowhere to put them
    assert call(mo=FAKE, ld=0) == 1
    assert call(mi=ctypes.c_void_p(4096), mo=ctypes.c_void_p(4096 + 64), ld=64) == 1   # overlap
    assert call(mo=ctypes.c_void_p(4100), ld=64) == 2
    assert cca.kernel_launches() == launches


def test_evict_refuses():
    L = cca.lib()
    launches = cca.kernel_launches()
    other = (5 << 24, 6 << 24, 7 << 24, 8 << 24)

    def call(a=None, b=None, lens=FAKE, mass=FAKE, ld=64, keep=16, recent=4, out=FAKE, mo=None, mld=0, slots=FAKE, ws=WS,
             n=BIG):
        a, b = a or cache(), b or cache(cap=32, ptrs=other)
        return L.attn_kv4_evict(ctypes.byref(a), lens, mass, ld, keep, recent, ctypes.byref(b), out, mo, mld, slots, ws, n,
                                None)

    for arg in ("lens", "mass", "out", "slots"):
        assert call(**{arg: None}) == 1
    assert call(keep=0) == 1 and call(keep=33) == 1 and call(recent=-1) == 1 and call(ld=0) == 1
    assert call(b=cache(cap=32)) == 1                                            # src and dst overlap
    assert call(b=cache(cap=32, ptrs=(5 << 24, 6 << 24, 7 << 24, (4 << 24) + 1008))) == 1
    assert call(b=cache(B=1, ptrs=other)) == 1 and call(b=cache(Hkv=1, ptrs=other)) == 1
    assert call(b=cache(D=128, ptrs=other)) == 1 and call(b=cache(ks=2.0, ptrs=other)) == 1
    assert call(mo=ctypes.c_void_p(1 << 30), mld=15) == 1
    assert call(mo=ctypes.c_void_p(4096 + 256), mld=16) == 1                    # mass and mass_out overlap
    assert call(ws=None) == 4
    assert cca.kernel_launches() == launches


def test_key_mass_refuses():
    L = cca.lib()
    launches = cca.kernel_launches()
    ch, n = _lib.chunk_array([(0, 256, 0, 0)])
    s = cca.make_shape(1, 2, 256, 64, 2 * 256 * 64, 64, 256 * 64, 0.125)

    def call(q=FAKE, k=FAKE, lse=FAKE, c=ch, nc=n, sh=s, mi=None, mo=FAKE, ws=WS, b=BIG):
        return L.attn_key_mass(q, k, lse, c, nc, ctypes.byref(sh), mi, mo, ws, b, None)

    for arg in ("q", "k", "lse", "mo"):
        assert call(**{arg: None}) == 1
    assert call(q=ctypes.c_void_p(4104)) == 2 and call(mo=ctypes.c_void_p(4100)) == 2
    assert call(ws=None) == 4 and call(b=0) == 4
    assert call(mi=ctypes.c_void_p(4096 + 256)) == 1                              # overlaps mass_out
    for bad in ([(0, 300, 0, 0)], [(0, 100, 0, 0), (50, 200, 0, 0)], [(10, 20, 11, 0)]):
        arr, m = _lib.chunk_array(bad)
        assert call(c=arr, nc=m) == 1
    assert call(sh=cca.make_shape(1, 2, 256, 100, 2 * 25600, 100, 25600, 0.1)) == 3
    assert cca.attn_workspace_size(s, [(0, 256, 0, 0)], cca.PASS_MASS) >= 256
    assert cca.attn_workspace_size(s, [], cca.PASS_MASS) >= 256
    assert cca.kernel_launches() == launches


def test_cache_object_checks_its_tensors():
    """Only layouts that the C description can express are accepted."""
    def arrays(B=2, Hkv=3, cap=32, D=80):
        return [torch.zeros((B, Hkv, cap, n), dtype=torch.uint8) for n in (D // 2, -(-D // 16)) * 2]

    c = cca.KV4Cache(*arrays(), D=80)
    assert (c.desc.sb, c.desc.sh, c.cap) == (96, 32, 32)
    big = arrays(B=4, Hkv=4, cap=64)
    v = cca.KV4Cache(*(t[1:3, ::2, :48] for t in big), D=80)
    assert (v.desc.sb, v.desc.sh, v.B, v.Hkv, v.cap) == (256, 128, 2, 2, 48)
    assert cca.KV4Cache(*(t[:1, :1] for t in big), D=80).desc.cap == 64
    for bad in ([t[:, :, ::2] for t in big],                                  # every other slot
                [t.transpose(1, 2) for t in big],                             # slots outermost
                [big[0][:2], *big[1:]],                                       # sizes differ
                [big[0][:, :2], *(t[:, ::2] for t in big[1:])],               # strides differ
                [t.float() for t in big]):
        with pytest.raises(cca.AttnError) as e:
            cca.KV4Cache(*bad, D=80)
        assert e.value.status == 1
    for D in (84, 0):
        with pytest.raises(cca.AttnError):
            cca.KV4Cache(*big, D=D)
    with pytest.raises(cca.AttnError) as e:
        cca.KV4Cache(*(t[:, :, :40] for t in big), D=80)                      # capacity not a multiple of 16
    assert e.value.status == 2


def test_wrappers_refuse_host_tensors_and_wrong_sizes():
    c = cca.kv4_cache(2, 2, 64, 64, device="cpu")
    x = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16)
    pos, ws = torch.zeros(2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    m = torch.zeros(2, 2, 64)
    for fn in (lambda: cca.kv4_store(c, x, x, pos, ws=ws), lambda: cca.kv4_load(c, pos, 3, ws=ws),
               lambda: cca.kv4_attention(x, c, pos, ws=ws), lambda: cca.kv4_attention(x, c, pos, mass_out=m, ws=ws),
               lambda: cca.kv4_evict(c, pos, m, 16, 4, cca.kv4_cache(2, 2, 32, 64, device="cpu"), ws=ws),
               lambda: cca.key_mass(x, x, torch.zeros(2, 2, 3), [(0, 3, 0, 0)], ws=ws)):
        with pytest.raises(cca.AttnError) as e:
            fn()
        assert e.value.status == 1


@pytest.mark.parametrize("cap,T,D", [(131072, 512, 128), (131072, 4096, 64), (262144, 64, 256), (1 << 20, 16, 128), (65536, 1 << 15, 128)])
def test_workspace_of_weights_is_bounded(cap, T, D):
    """Scores of all rows of a long call would take up to 550 GB; what is kept stays within 1 GiB or a group of rows."""
    c = cache(B=1, Hkv=8, cap=cap, D=D)
    s = cca.make_shape(1, 32, T, D, 32 * T * D, D, T * D, 0.125)
    plain = cca.attn_kv4_workspace_size(c, s, cca.KV4_ATTEND)
    group = 4 * 8 * cap * (32 if D <= 128 else 16)
    lse = 4 * 32 * T + 256
    assert cca.attn_kv4_workspace_size(c, s, cca.KV4_ATTEND_MASS) <= plain + lse + max(1 << 30, group)


@pytest.mark.parametrize("B,Hkv,cap,sb,sh,ok", [
    (2, 2, 64, 128, 64, True), (2, 2, 64, 64, 128, True), (3, 4, 32, 32, 96, True), (3, 4, 32, 128, 32, True),
    (2, 3, 48, 640, 64, True), (2, 3, 48, 64, 640, True), (2, 1, 64, 64, 16, True), (1, 2, 64, 16, 64, True),
    (2, 2, 64, 64, 64, False),                      # head 1 of sequence 0 is head 0 of sequence 1
    (2, 2, 64, 112, 64, False), (3, 3, 32, 64, 32, False), (2, 4, 64, 128, 64, False), (4, 2, 64, 64, 128, False),
    (2, 2, 64, 1 << 62, 64, False), (2, 2, 64, 64, 1 << 62, False)])
def test_cache_rows_are_not_shared(B, Hkv, cap, sb, sh, ok):
    """Two rows of a cache in the same place: a store would write both."""
    rows = {b * sb + h * sh + t for b in range(B) for h in range(Hkv) for t in range(cap)}
    assert not ok or len(rows) == B * Hkv * cap
    c = cache(B=B, Hkv=Hkv, cap=cap, sb=sb, sh=sh)
    n = ctypes.c_size_t(0)
    assert cca.lib().attn_kv4_workspace_size(ctypes.byref(c), None, 0, ctypes.byref(n)) == (0 if ok else 1)


def test_cache_object_refuses_shared_rows():
    a = [torch.zeros(4 * 64, n, dtype=torch.uint8) for n in (32, 4, 32, 4)]
    shared = [t.as_strided((2, 2, 64, n), (64 * n, 64 * n, n, 1)) for t, n in zip(a, (32, 4, 32, 4))]
    with pytest.raises(cca.AttnError) as e:
        cca.KV4Cache(*shared, D=64)
    assert e.value.status == 1


def test_evict_within_one_allocation():
    """Source and destination are slots of the same larger cache: between one another, or overlapping."""
    L = cca.lib()

    def call(a, b, mass=1 << 40, ld=256, mo=None, mld=0, B=2, Hkv=2, **kw):
        view = lambda first, cap: cache(B=B, Hkv=Hkv, cap=cap, sb=Hkv * 256, sh=256,
                                        ptrs=[(i << 24) + first * n for i, n in ((1, 32), (2, 4), (3, 32), (4, 4))])
        # a missing workspace (4) is seen after the overlaps (1)
        return L.attn_kv4_evict(ctypes.byref(view(*a)), FAKE, ctypes.c_void_p(mass), ld, 16, 4, ctypes.byref(view(*b)), FAKE,
                                mo and ctypes.c_void_p(mo), mld, FAKE, None, 0, None)

    for B, Hkv in ((2, 2), (1, 2), (2, 1), (1, 1)):
        assert call((0, 128), (128, 128), B=B, Hkv=Hkv) == 4 and call((128, 64), (64, 64), B=B, Hkv=Hkv) == 4
        assert call((0, 128), (112, 64), B=B, Hkv=Hkv) == 1 and call((0, 128), (0, 32), B=B, Hkv=Hkv) == 1
        assert call((64, 64), (32, 48), B=B, Hkv=Hkv) == 1
    assert call((0, 144), (240, 32)) == 1                  # its last slots are the next head's first
    # rows of weights between one another: 128 in, 16 out, 256 apart
    assert call((0, 128), (128, 128), mo=(1 << 40) + 4 * 128, mld=256) == 4
    assert call((0, 128), (128, 128), mo=(1 << 40) - 4 * 128, mld=256) == 4
    assert call((0, 128), (128, 128), mo=(1 << 40) + 4 * 124, mld=256) == 1
    assert call((0, 128), (128, 128), mo=(1 << 40) + 4 * 128, mld=192) == 1      # not at the same distance
    assert call((0, 128), (128, 128), ld=1 << 62) == 1


def test_weights_of_a_call_between_one_another():
    L, s, c = cca.lib(), shape(), cache(cap=64)
    call = lambda mi, mo, ld: L.attn_kv4_attend(FAKE, ctypes.byref(s), ctypes.byref(c), FAKE, FAKE, FAKE, ctypes.c_void_p(mi),
                                                ctypes.c_void_p(mo), ld, None, 0, None)
    assert call(1 << 40, (1 << 40) + 256, 128) == 4 and call((1 << 40) + 256, 1 << 40, 128) == 4
    assert call(1 << 40, 1 << 40, 128) == 4
    assert call(1 << 40, (1 << 40) + 240, 128) == 1 and call(1 << 40, (1 << 40) + 272, 128) == 1
    assert call(1 << 40, 1 << 41, 1 << 62) == 1


@pytest.mark.parametrize("B,H,T,sb,sh,st,ok", [
    (2, 2, 3, 384, 192, 64, True), (2, 2, 3, 384, 64, 128, True), (2, 2, 3, 64, 128, 256, True), (2, 2, 3, 4096, 72, 160, True),
    (2, 2, 1, 128, 64, 8, True), (2, 2, 3, 384, 192, 56, False), (2, 2, 3, 384, 64, 64, False), (2, 2, 3, 320, 192, 64, False),
    (2, 2, 3, 256, 128, 64, False), (2, 2, 3, 1 << 62, 1 << 62, 1 << 62, False)])
def test_rows_that_are_written_lie_apart(B, H, T, sb, sh, st, ok):
    """Queries' strides are the outputs' too: windows that overlap would be written twice. Rows to store may overlap."""
    s, c, L = cca.make_shape(B, H, T, 64, sb, st, sh, 0.125), cache(B=B, Hkv=H, cap=64), cca.lib()
    # a missing workspace (4) is seen after the strides (1)
    want = 4 if ok else 1
    assert L.attn_kv4_attend(FAKE, ctypes.byref(s), ctypes.byref(c), FAKE, FAKE, FAKE, None, None, 0, None, 0, None) == want
    assert L.attn_kv4_load(ctypes.byref(c), FAKE, None, ctypes.byref(s), FAKE, FAKE, None, 0, None) == want
    assert L.attn_kv4_store(FAKE, FAKE, ctypes.byref(s), ctypes.byref(c), FAKE, None, None, 0, None) == 4
