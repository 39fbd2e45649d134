"""GPU parity of the 4-bit key/value cache and of the key mass with the float64
oracle (oracle.kv4).

Tolerances, derived from the arithmetic (eps of the last place, relative):
  * Stored codes and scales, evicted slots: equal.
  * A score is a sum of D products that are exact, in fp32: each of at most D
    additions is off by at most 2^-23 of the sum of magnitudes (a tensor core may
    truncate), and scaling it to base 2 by 2^-23 of itself twice. With A the largest
    sum of magnitudes |q||k| scale of a call: e = (D + 4) 2^-23 A. ex2.approx is off by
    2^-22, an accumulated sum of at most n weights in fp32, in partial sums of no more
    than 2^10 terms each, by 2^10 2^-24.
  * A weight is rounded to fp16's 11 bits: 2^-11 of itself, or is flushed below 2^-35 of
    the row's largest.
  * O is the weighted sum of |v| with those errors, rounded to bf16 (2^-8).
"""
import math
import os

import numpy as np
import pytest
import torch

import chunked_causal_attention_gb300 as cca
from oracle import kv4 as K

from parity import head, lse_head

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
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(x):
    return x.detach().double().cpu().numpy()


def bf16(rng, *shape):
    return torch.tensor(rng.normal(size=shape), dtype=torch.float32).bfloat16().cuda()


def random_cache(B, Hkv, cap, D, seed, ts=(0.5, 2.0), view=False):
    """A cache of random codes and scales between 2^-5 and 2, as a view of a larger one if asked;
    slots hold NaN scales where the test does not overwrite them."""
    rng = np.random.default_rng(seed)
    B2, H2, cap2 = (B + 1, Hkv + 1, cap + 16) if view else (B, Hkv, cap)
    nb = -(-D // 16)
    arrays = []
    for _ in range(2):
        arrays.append(torch.tensor(rng.integers(0, 256, (B2, H2, cap2, D // 2)), dtype=torch.uint8).cuda())
        arrays.append(torch.tensor(rng.integers(0x10, 0x40, (B2, H2, cap2, nb)), dtype=torch.uint8).cuda())
    if view:
        arrays = [a[1:, 1:, :cap] for a in arrays]
    return cca.KV4Cache(*arrays, D=D, k_scale=ts[0], v_scale=ts[1])


def cached(c, b, h, n):
    """Float64 (k, v) of the first n slots."""
    g = lambda t: t[b, h, :n].cpu().numpy()
    return (K.values(g(c.k_codes), g(c.k_scales), c.k_scale), K.values(g(c.v_codes), g(c.v_scales), c.v_scale))


def score_error(q, k, scale):
    """Error bound of a base-2 score and its weight's relative error (see the header)."""
    a = (np.abs(q) @ np.abs(k).T).max() * abs(scale) if k.size else 0.0
    return (q.shape[-1] + 4) * 2.0 ** -23 * a + 2.0 ** -21


def check_attend(q, c, lens, o, lse, scale=None, mass_in=None, mass_out=None, kept_tail=None):
    B, H, T, D = q.shape
    G = H // c.Hkv
    sc = 1.0 / math.sqrt(D) if scale is None else scale
    for b in range(B):
        n = int(lens[b])
        for hk in range(c.Hkv):
            k, v = cached(c, b, hk, n)
            qs = f64(q[b, hk * G:(hk + 1) * G])
            ro, rl, w = K.attend(qs, k, v, n, sc)
            e = score_error(qs, k, sc)
            go, gl = f64(o[b, hk * G:(hk + 1) * G]), f64(lse[b, hk * G:(hk + 1) * G])
            assert (np.isneginf(gl) == np.isneginf(rl)).all()
            ok = np.isfinite(rl)
            assert (np.abs(gl[ok] - rl[ok]) <= e + SUM + 2.0 ** -22 * (1 + np.abs(rl[ok]))).all(), np.abs(gl[ok] - rl[ok]).max()
            wv = w @ np.abs(v)                                       # sum of weight * |v|
            tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2 * e + 2 * SUM) * wv + 2.0 ** -35 * max(n, 1) * (np.abs(v).max() if n else 0)
            assert (np.abs(go - ro) <= tol + 1e-30).all(), (b, hk, (np.abs(go - ro) / (tol + 1e-30)).max())
            if mass_out is not None:
                ref = w.sum((0, 1)) + (f64(mass_in[b, hk, :n]) if mass_in is not None else 0.0)
                got = f64(mass_out[b, hk])
                tol = (2 * e + 2 * SUM) * w.sum((0, 1)) + 2.0 ** -22 * ref
                assert (np.abs(got[:n] - ref) <= tol + 1e-35).all(), (np.abs(got[:n] - ref) / (tol + 1e-35)).max()
                if kept_tail is not None:
                    assert (got[n:] == kept_tail).all()


# ------------------------------------------------------------------ rows

def special_rows(rng, *shape):
    """Normal rows with blocks of zeros, ties, tiny and huge values, infinities and NaN."""
    x = torch.tensor(rng.normal(size=shape) * np.exp2(rng.integers(-12, 10, shape[:-1] + (1,)))).bfloat16()
    flat = x.view(-1, shape[-1])
    for i in range(0, flat.shape[0], 2):
        kind, a = i // 2 % 8, 0 if shape[-1] < 24 else 16
        n = min(16, shape[-1] - a)
        if kind == 0:
            flat[i, a:a + n] = 0.0
        elif kind == 1:
            flat[i, a:a + n] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -0.0][:n])
        elif kind == 2:
            flat[i, a] = float("inf")
        elif kind == 3:
            flat[i, a + 1] = float("nan")
        elif kind == 4:
            flat[i, a:a + n] *= 1e-38
        elif kind == 5:
            flat[i, a:a + n] *= 1e30
        elif kind == 6:
            flat[i, a:a + n] = 6.375 * torch.tensor([1.0, -0.5] * 8)[:n]
        else:
            flat[i, a] = -float("inf")
    return x


def expected_rows(x, ts):
    codes, scales = zip(*(K.quantise_row(r, ts) for r in x.reshape(-1, x.shape[-1]).double().numpy()))
    return (np.stack(codes).reshape(x.shape[:-1] + (-1,)), np.stack(scales).reshape(x.shape[:-1] + (-1,)))


@pytest.mark.parametrize("D", [8, 16, 40, 64, 80, 128, 136, 256])
@pytest.mark.parametrize("T,ts", [(1, (1.0, 1.0)), (21, (0.25, 8.0))])
def test_store_and_load_dense(D, T, ts):
    rng = np.random.default_rng(D + T)
    B, Hkv, cap = 3, 2, 48
    c = cca.kv4_cache(B, Hkv, cap, D, k_scale=ts[0], v_scale=ts[1])
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.fill_(0xAB)
    k, v = special_rows(rng, B, Hkv, T, D), special_rows(rng, B, Hkv, T, D)
    pos = [0, 5, cap - T]
    ws = cca.kv4_workspace(c)
    # token-major storage of the inputs
    kd, vd = (x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) for x in (k, v))
    cca.kv4_store(c, kd, vd, i32(pos), ws=ws)
    lk, lv = cca.kv4_load(c, i32(pos), T, ws=ws)
    assert cca.attn_status(ws) == 0
    for x, got, codes, scales, s in ((k, lk, c.k_codes, c.k_scales, ts[0]), (v, lv, c.v_codes, c.v_scales, ts[1])):
        ec, es = expected_rows(x, s)
        want = torch.tensor(K.values(ec, es, s)).to(torch.bfloat16)
        assert torch.equal(got.cpu().view(torch.int16)[~want.isnan()], want.view(torch.int16)[~want.isnan()])
        assert torch.equal(got.cpu().isnan(), want.isnan())
        for b in range(B):
            rows = slice(pos[b], pos[b] + T)
            assert (codes[b, :, rows].cpu().numpy() == ec[b]).all() and (scales[b, :, rows].cpu().numpy() == es[b]).all()
            rest = torch.ones(cap, dtype=torch.bool)
            rest[rows] = False
            assert (codes[b].cpu()[:, rest] == 0xAB).all() and (scales[b].cpu()[:, rest] == 0xAB).all()


@pytest.mark.parametrize("D,lens", [(64, [3, 0, 1, 17, 0]), (80, [5, 1, 1, 1, 30])])
def test_store_and_load_packed(D, lens):
    rng = np.random.default_rng(D)
    B, Hkv, cap = len(lens), 3, 32
    cu = np.concatenate(([0], np.cumsum(lens)))
    c = cca.kv4_cache(B, Hkv, cap, D)
    k, v = bf16(rng, cu[-1], Hkv, D), bf16(rng, cu[-1], Hkv, D)
    pos = [2, 0, 31, 0, 1]
    ws = cca.kv4_workspace(c)
    cca.kv4_store(c, k, v, i32(pos), cu_seqlens=i32(cu.tolist()), ws=ws)
    lk, lv = cca.kv4_load(c, i32(pos), int(cu[-1]), cu_seqlens=i32(cu.tolist()), ws=ws)
    assert cca.attn_status(ws) == 0
    for x, got, codes, scales in ((k, lk, c.k_codes, c.k_scales), (v, lv, c.v_codes, c.v_scales)):
        ec, es = expected_rows(x.cpu(), 1.0)
        assert (f64(got) == K.values(ec, es, 1.0)).all()
        for b in range(B):
            assert (codes[b, :, pos[b]:pos[b] + lens[b]].cpu().numpy() == ec[cu[b]:cu[b + 1]].swapaxes(0, 1)).all()
        assert int((scales != 0).sum()) == int((es != 0).sum())          # nothing else was written


def test_rows_outside_the_cache_are_skipped_and_reported():
    rng = np.random.default_rng(3)
    c = cca.kv4_cache(4, 1, 16, 64)
    k, v = bf16(rng, 4, 1, 3, 64), bf16(rng, 4, 1, 3, 64)
    ws = cca.kv4_workspace(c)
    pos = i32([-1, 14, 2 ** 31 - 2, 3])
    cca.kv4_store(c, k, v, pos, ws=ws)
    assert cca.attn_status(ws) == 7 and cca.attn_status(ws) == 0
    used = c.k_scales.ne(0).any(-1).cpu()[:, 0]
    assert [r.nonzero().flatten().tolist() for r in used] == [[0, 1], [14, 15], [], [3, 4, 5]]
    out = torch.full_like(k, 7.0)
    lk, _ = cca.kv4_load(c, pos, 3, k=out, v=torch.empty_like(v), ws=ws)
    assert cca.attn_status(ws) == 7
    assert (lk[0, 0, 0] == 7).all() and (lk[1, 0, 2] == 7).all() and (lk[2] == 7).all() and not (lk[3] == 7).any()
    # packed: tokens before the first offset and after the last belong to no sequence
    c2 = cca.kv4_cache(2, 1, 16, 64)
    p = k.reshape(12, 1, 64)
    cca.kv4_store(c2, p, p, i32([0, 0]), cu_seqlens=i32([1, 4, 6]), ws=ws)
    assert cca.attn_status(ws) == 7
    assert c2.k_scales.ne(0).any(-1).sum(-1).flatten().tolist() == [3, 2]


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("D", [8, 40, 64, 80, 128, 136, 200, 256])
@pytest.mark.parametrize("G,T", [(1, 1), (4, 1), (5, 3), (8, 1), (3, 11), (16, 4)])
def test_attend(D, G, T):
    B, Hkv, cap = 5, 2, 272
    rng = np.random.default_rng(D + 7 * G + T)
    c = random_cache(B, Hkv, cap, D, D + G, view=True)
    lens = [0, 1, 130, 257, cap]
    # slots behind the last one in use hold NaN
    for b, n in enumerate(lens):
        c.k_scales[b, :, n:] = 0x7F
        c.v_scales[b, :, n:] = 0xFF
    q = 2 * bf16(rng, B, Hkv * G, T, D)
    ws = cca.kv4_workspace(c, q, mass=True)
    o, lse = cca.kv4_attention(q, c, i32(lens), ws=ws)
    check_attend(q, c, lens, o, lse)
    mi, mo = torch.rand(B, Hkv, cap, device="cuda"), torch.full((B, Hkv, cap), -3.0, device="cuda")
    o2, lse2 = cca.kv4_attention(q, c, i32(lens), mass_in=mi, mass_out=mo, ws=ws)
    assert cca.attn_status(ws) == 0
    check_attend(q, c, lens, o2, lse2, None, mi, mo, kept_tail=-3.0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # in place, and from nothing
    m = mi.clone()
    cca.kv4_attention(q, c, i32(lens), mass_in=m, mass_out=m, ws=ws)
    for b, n in enumerate(lens):
        assert torch.equal(m[b, :, :n], mo[b, :, :n]) and torch.equal(m[b, :, n:], mi[b, :, n:])
    mo.fill_(0)
    cca.kv4_attention(q, c, i32(lens), mass_out=mo, ws=ws)
    check_attend(q, c, lens, o, lse, None, None, mo, kept_tail=0.0)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000, 4095, 4096])
def test_attend_lengths(n):
    c = random_cache(1, 3, 4096, 128, n)
    q = 2 * bf16(np.random.default_rng(n), 1, 12, 1, 128)
    o, lse = cca.kv4_attention(q, c, i32([n]))
    check_attend(q, c, [n], o, lse)


def test_attend_many_ragged_sequences():
    rng = np.random.default_rng(17)
    lens = [int(x) for x in rng.integers(0, 500, 70)]
    c = random_cache(70, 2, 512, 64, 18)
    q = bf16(rng, 70, 8, 2, 64)
    mo = torch.zeros(70, 2, 512, device="cuda")
    o, lse = cca.kv4_attention(q, c, i32(lens), scale=0.3, mass_out=mo)
    check_attend(q, c, lens, o, lse, 0.3, None, mo, kept_tail=0.0)


def test_attend_long_with_split_keys():
    """One key/value head over 100,003 slots: its keys are spread over many blocks."""
    n, D = 100003, 128
    c = random_cache(1, 1, 100016, D, 4)
    q = 3 * bf16(np.random.default_rng(5), 1, 4, 1, D)
    mo = torch.zeros(1, 1, 100016, device="cuda")
    o, lse = cca.kv4_attention(q, c, i32([n]), mass_out=mo)
    check_attend(q, c, [n], o, lse, None, None, mo)


def test_attend_more_sequences_than_threads():
    """300 sequences, most of them empty: blocks find theirs by a scan over more than one group."""
    rng = np.random.default_rng(19)
    lens = [int(x) if x % 3 == 0 else 0 for x in rng.integers(0, 200, 300)]
    lens[-1] = 208
    c = random_cache(300, 1, 208, 64, 20)
    q = bf16(rng, 300, 2, 1, 64)
    o, lse = cca.kv4_attention(q, c, i32(lens))
    check_attend(q, c, lens, o, lse)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-3])
def test_attend_many_rows_and_scales(scale):
    """A prompt chunk's worth of rows, more than there are slots, at scales other than 1/sqrt(D)."""
    rng = np.random.default_rng(27)
    c = random_cache(1, 2, 272, 80, 28)
    q = bf16(rng, 1, 6, 300, 80)
    mo = torch.zeros(1, 2, 272, device="cuda")
    o, lse = cca.kv4_attention(q, c, i32([257]), scale=scale, mass_out=mo)
    check_attend(q, c, [257], o, lse, scale, None, mo, kept_tail=0.0)


def test_offsets_past_32_bits():
    """Heads 70 million slots apart: byte offsets of the second head pass 2^32."""
    apart, cap, D = 70_000_000 // 16 * 16, 512, 128
    arrays = [torch.empty((1, 2, apart, n), dtype=torch.uint8, device="cuda")[:, :, :cap] for n in (64, 8, 64, 8)]
    c = cca.KV4Cache(*arrays, D=D)
    assert c.desc.sh * 64 > 1 << 32
    rng = np.random.default_rng(29)
    k, v = bf16(rng, 1, 2, cap, D), bf16(rng, 1, 2, cap, D)
    cca.kv4_store(c, k, v, i32([0]))
    kk, vv = cca.kv4_load(c, i32([0]), cap)
    near = cca.kv4_cache(1, 2, cap, D)
    cca.kv4_store(near, k, v, i32([0]))
    nk, nv = cca.kv4_load(near, i32([0]), cap)
    assert torch.equal(kk, nk) and torch.equal(vv, nv)
    q = bf16(rng, 1, 8, 2, D)
    for a, b in zip(cca.kv4_attention(q, c, i32([500])), cca.kv4_attention(q, near, i32([500]))):
        assert torch.equal(a, b)
    mass = torch.rand(1, 2, cap, device="cuda")
    small = [cca.kv4_cache(1, 2, 64, D) for _ in range(2)]
    for s, x in zip(small, (c, near)):
        cca.kv4_evict(x, i32([500]), mass, 64, 8, s)
    assert torch.equal(small[0].v_codes, small[1].v_codes) and torch.equal(small[0].k_scales, small[1].k_scales)


@pytest.mark.parametrize("window", [False, True])
def test_waits_that_run_out_are_reported(monkeypatch, window):
    """With the copies held back (a test switch) every wait ends after its limit with ATTN_E_TIMEOUT in the
    status word, and the next calls work."""
    rng = np.random.default_rng(30)
    c = random_cache(1, 1, 256, 64, 31)
    q = bf16(rng, 1, 2, 1, 64)
    ws = cca.kv4_workspace(c, q)
    good, _ = cca.kv4_attention(q, c, i32([250]), ws=ws)
    qq, k = bf16(rng, 1, 2, 700, 64), bf16(rng, 1, 1, 700, 64)
    chunks = [(690, 700, 0, 0)] if window else [(0, 700, 0, 0)]
    _, lse = cca.forward(qq, k, k, chunks)
    mws = cca.key_mass_workspace(qq, k, chunks)
    want = cca.key_mass(qq, k, lse, chunks, ws=mws)
    monkeypatch.setenv("ATTN_TEST_STALL_PRODUCER", "1")
    monkeypatch.setenv("ATTN_WAIT_LIMIT_MS", "200")
    cca.kv4_attention(q, c, i32([250]), ws=ws)
    assert cca.attn_status(ws) == 6
    cca.key_mass(qq, k, lse, chunks, ws=mws)
    assert cca.attn_status(mws) == 6
    monkeypatch.delenv("ATTN_TEST_STALL_PRODUCER")
    assert torch.equal(cca.kv4_attention(q, c, i32([250]), ws=ws)[0], good)
    assert torch.equal(cca.key_mass(qq, k, lse, chunks, ws=mws), want)
    assert cca.attn_status(ws) == 0 and cca.attn_status(mws) == 0


def test_attend_strided_queries_and_repeat():
    """Token-major queries, a view of wider rows, scores of one sharp maximum; the same bits each time."""
    rng = np.random.default_rng(9)
    c = random_cache(2, 2, 512, 80, 10)
    q = (20 * bf16(rng, 2, 3, 8, 128)).permute(0, 2, 1, 3)[..., :80]
    lens = [512, 77]
    o, lse = cca.kv4_attention(q, c, i32(lens))
    assert o.stride() == q.stride()
    check_attend(q, c, lens, o, lse)
    for _ in range(5):
        o2, lse2 = cca.kv4_attention(q, c, i32(lens))
        assert torch.equal(o2, o) and torch.equal(lse, lse2)


def test_attend_extreme_queries():
    """Zero, smallest and largest bf16 queries: the power-of-two scaling keeps their scores; an
    infinite or NaN query gives NaN in its own row only."""
    c = random_cache(1, 1, 64, 64, 11)
    q = torch.zeros(1, 6, 1, 64, device="cuda", dtype=torch.bfloat16)
    q[0, 1] = 1e-40
    q[0, 2] = bf16(np.random.default_rng(1), 1, 64) * 1e-30
    q[0, 3] = bf16(np.random.default_rng(2), 1, 64) * 1e30
    q[0, 4, 0, 3] = float("inf")
    q[0, 5, 0, 7] = float("nan")
    o, lse = cca.kv4_attention(q, c, i32([64]), scale=1.0)
    check_attend(q[:, :3], c, [64], o[:, :3], lse[:, :3], 1.0)
    k, v = cached(c, 0, 0, 64)
    s = f64(q[0, 3]) @ k.T
    best = s[0].argmax()
    assert np.allclose(f64(o[0, 3, 0]), v[best], rtol=2.0 ** -8) and np.isclose(f64(lse[0, 3, 0]), s[0].max(), rtol=1e-5)
    assert o[0, 4:].isnan().all() and lse[0, 4:].isnan().all()


@pytest.mark.parametrize("D", [64, 80, 128, 256])
def test_attend_nan_rows(D):
    """A slot whose keys or values are NaN reaches the queries that see it and no other."""
    T, n = 4, 150
    for what in ("k", "v"):
        c = random_cache(1, 1, 160, D, 12)
        blk = -(-D // 16) // 2
        getattr(c, what + "_scales")[0, 0, n - 2, blk] = 0x7F          # seen by queries T-2 and T-1
        q = bf16(np.random.default_rng(13), 1, 2, T, D)
        o, lse = cca.kv4_attention(q, c, i32([n]))
        bad = o[0, :, T - 2:].isnan()
        if what == "k":
            assert bad.all() and lse[0, :, T - 2:].isnan().all()
        else:
            hit = torch.zeros(D, dtype=torch.bool, device="cuda")
            hit[16 * blk:16 * blk + 16] = True
            assert (bad == hit).all() and lse.isfinite().all()
        assert o[0, :, :T - 2].isfinite().all() and lse[0, :, :T - 2].isfinite().all()


def test_attend_reports_bad_lengths():
    c = random_cache(3, 1, 64, 64, 14)
    q = bf16(np.random.default_rng(15), 3, 2, 1, 64)
    ws = cca.kv4_workspace(c, q, mass=True)
    o, lse = cca.kv4_attention(q, c, i32([65, -1, 64]), ws=ws)
    good, gl = cca.kv4_attention(q, c, i32([64, 0, 64]))
    assert cca.attn_status(ws) == 7 and torch.equal(o, good) and torch.equal(lse, gl)
    mo = torch.zeros(3, 1, 40, device="cuda")
    o, _ = cca.kv4_attention(q, c, i32([41, 40, 3]), mass_out=mo, ws=ws)
    want, _ = cca.kv4_attention(q, c, i32([40, 40, 3]))
    assert cca.attn_status(ws) == 7 and torch.equal(o, want)


# ------------------------------------------------------------------ key mass

def check_mass(q, k, lse, chunks, got, scale, mass_in=None, packed=False):
    Hkv = k.shape[1]
    B, H = (1, q.shape[1]) if packed else q.shape[:2]
    G = H // Hkv
    for b in range(B):
        for hk in range(Hkv):
            hs = range(hk * G, hk * G + G)
            qs = np.stack([head(q, b, h, packed) for h in hs])
            ls = np.stack([lse_head(lse, b, h) for h in hs])
            kh = head(k, b, hk, packed)
            ref = K.key_mass(qs, kh, ls, chunks, scale)
            e = score_error(qs.reshape(-1, qs.shape[-1]), kh, scale) + 2.0 ** -22 * np.abs(ls[np.isfinite(ls)]).max(initial=0)
            base = f64(mass_in[b, hk]) if mass_in is not None else 0.0
            tol = (2 * e + SUM) * ref + 2.0 ** -22 * np.abs(base + ref) + 1e-35
            d = np.abs(f64(got[b, hk]) - base - ref)
            assert (d <= tol).all(), (b, hk, int((d / tol).argmax()), (d / tol).max())


MASS_PLANS = {"whole": [(0, 700, 0, 0)], "cut": [(0, 300, 0, 0), (300, 301, 0, 0), (301, 700, 0, 128)],
              "window": [(683, 700, 0, 0)], "one row": [(699, 700, 0, 0)], "gap": [(0, 130, 0, 0), (500, 650, 0, 0)],
              "docs": [(0, 257, 0, 0), (257, 258, 257, 0), (258, 700, 258, 0)],
              "late context": [(300, 500, 250, 0), (600, 700, 599, 0)], "late window": [(600, 640, 333, 0)],
              "early window": [(128, 140, 0, 0)], "none": []}


@pytest.mark.parametrize("plan", list(MASS_PLANS))
@pytest.mark.parametrize("D,H,Hkv", [(128, 4, 4), (64, 6, 2), (80, 4, 1), (256, 2, 1), (8, 3, 3)])
def test_key_mass(plan, D, H, Hkv):
    rng = np.random.default_rng(D + H)
    L, chunks = 700, MASS_PLANS[plan]
    q, k, v = 2 * bf16(rng, 2, H, L, D), bf16(rng, 2, Hkv, L, D), bf16(rng, 2, Hkv, L, D)
    lse = torch.zeros(2, H, L, device="cuda")
    if chunks:
        _, lse = cca.forward(q, k, v, chunks)
    got = cca.key_mass(q, k, lse, chunks)
    check_mass(q, k, lse, chunks, got, D ** -0.5)
    assert torch.equal(got, cca.key_mass(q, k, lse, chunks))
    m = torch.rand(2, Hkv, L, device="cuda")
    start = m.clone()
    out = cca.key_mass(q, k, lse, chunks, mass_in=m, mass_out=m)
    assert out is m
    check_mass(q, k, lse, chunks, m, D ** -0.5, mass_in=start)


@pytest.mark.parametrize("L", [1, 2, 127, 128, 129, 255, 256, 257, 1500])
def test_key_mass_lengths_and_total(L):
    rng = np.random.default_rng(L)
    q, k = 2 * bf16(rng, 1, 2, L, 128), bf16(rng, 1, 1, L, 128)
    _, lse = cca.forward(q, k, k, [(0, L, 0, 0)])
    got = cca.key_mass(q, k, lse, [(0, L, 0, 0)])
    check_mass(q, k, lse, [(0, L, 0, 0)], got, 128 ** -0.5)
    # every row's weights sum to one; lse and the sums are good to a few 2^-20
    assert abs(float(got.double().sum()) - 2 * L) <= 2 * L * 1e-4


def test_key_mass_packed_streamed_and_empty_rows():
    """Packed documents, one call per chunk accumulating in place, and rows without a log-sum-exp."""
    rng = np.random.default_rng(31)
    cu = [0, 100, 101, 400, 640]
    q, k, v = 2 * bf16(rng, 640, 4, 64), bf16(rng, 640, 2, 64), bf16(rng, 640, 2, 64)
    chunks = cca.attn_plan_varlen(cu, 256, cca.PLAN_UNIFORM)
    _, lse = cca.forward(q, k, v, chunks, packed=True)
    got = cca.key_mass(q, k, lse, chunks, packed=True)
    check_mass(q, k, lse, chunks, got, 0.125, packed=True)
    m = torch.zeros(1, 2, 640, device="cuda")
    ws = cca.key_mass_workspace(q, k, chunks, packed=True)
    for c in chunks:
        cca.key_mass(q, k, lse, [c], packed=True, mass_in=m, mass_out=m, ws=ws)
    assert cca.attn_status(ws) == 0
    check_mass(q, k, lse, chunks, m, 0.125, packed=True)
    lse[0, :, 50:90] = -math.inf
    check_mass(q, k, lse, chunks, cca.key_mass(q, k, lse, chunks, packed=True), 0.125, packed=True)


@pytest.mark.parametrize("D,H,Hkv,w", [(128, 6, 3, 40), (128, 16, 2, 64), (64, 9, 3, 100), (256, 3, 3, 128), (80, 8, 1, 1),
                                        (128, 4, 4, 129), (40, 8, 2, 17)])
def test_key_mass_of_a_window(D, H, Hkv, w):
    """Few rows over many key tiles: several tiles, and the ends of heads, in one block of the grid."""
    rng = np.random.default_rng(D + w)
    L = 19000 + w
    q, k = 2 * bf16(rng, 1, H, L, D), bf16(rng, 1, Hkv, L, D)
    chunks = [(L - w - 1, L - 1, 0, 0)]                        # the last key is seen by no row
    _, lse = cca.forward(q, k, k, chunks)
    lse[0, 0, L - 2] = -math.inf                               # a row that counts for nothing
    got = cca.key_mass(q, k, lse, chunks)
    check_mass(q, k, lse, chunks, got, D ** -0.5)
    assert (got[..., -1] == 0).all() and torch.equal(got, cca.key_mass(q, k, lse, chunks))
    m = torch.rand(1, Hkv, L, device="cuda")
    check_mass(q, k, lse, chunks, cca.key_mass(q, k, lse, chunks, mass_in=m), D ** -0.5, mass_in=m)


@pytest.mark.parametrize("D,G", [(64, 1), (80, 2), (128, 1)])
@pytest.mark.parametrize("chunks", [[(0, 1300, 0, 0)], [(0, 257, 0, 0), (257, 390, 257, 0), (390, 1300, 390, 0)],
                                    [(0, 130, 0, 0), (600, 1290, 100, 0)], [(700, 1300, 128, 0)]])
def test_key_mass_with_many_heads(D, G, chunks):
    """Many heads and key tiles of few blocks: the groups that sum skip items in which they have none."""
    rng = np.random.default_rng(D + G)
    B, Hkv, L = 2, 64, 1300
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    q = 2 * torch.randn(B, Hkv * G, L, D, device="cuda", generator=g).bfloat16()
    k = torch.randn(B, Hkv, L, D, device="cuda", generator=g).bfloat16()
    _, lse = cca.forward(q, k, k, chunks)
    got = cca.key_mass(q, k, lse, chunks)
    heads = [0, 1, 31, 63]
    qs = [h * G + i for h in heads for i in range(G)]
    check_mass(q[:, qs], k[:, heads], lse[:, qs], chunks, got[:, heads], D ** -0.5)
    # the other heads by the sum of their weights: one a row
    total = G * sum(b - a for a, b, _, _ in chunks)
    assert (got.double().sum(-1) - total).abs().max() <= total * 1e-4
    for _ in range(3):
        assert torch.equal(got, cca.key_mass(q, k, lse, chunks))
    m = torch.rand(B, Hkv, L, device="cuda")
    out = cca.key_mass(q, k, lse, chunks, mass_in=m)
    check_mass(q[:, qs], k[:, heads], lse[:, qs], chunks, out[:, heads], D ** -0.5, mass_in=m[:, heads])


def test_key_mass_strided():
    """Token-major storage, 80 dims of a wider buffer, a batch view."""
    rng = np.random.default_rng(33)
    q = bf16(rng, 3, 200, 4, 128).permute(0, 2, 1, 3)[1:, ..., :80]
    k = bf16(rng, 3, 200, 2, 96).permute(0, 2, 1, 3)[1:, ..., :80]
    chunks = [(0, 200, 0, 0)]
    _, lse = cca.forward(q, k, k, chunks)
    check_mass(q, k, lse, chunks, cca.key_mass(q, k, lse, chunks), 80 ** -0.5)


# ------------------------------------------------------------------ eviction

MASSES = {
    "spread": lambda rng, s: np.exp(2 * rng.normal(size=s)),
    "ties": lambda rng, s: rng.integers(0, 4, s).astype(np.float64),
    "equal": lambda rng, s: np.ones(s),
    "special": lambda rng, s: rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, -1.5, 1e-40, -1e-40, 3.0], s),
}


@pytest.mark.parametrize("kind", list(MASSES))
@pytest.mark.parametrize("keep,recent,D", [(1, 0, 64), (100, 0, 128), (100, 30, 40), (64, 64, 256), (33, 500, 8),
                                           (512, 3, 128)])
def test_evict(kind, keep, recent, D):
    rng = np.random.default_rng(keep + recent)
    B, Hkv, cap = 5, 2, 512
    lens = [0, 1, keep, 300, cap]
    src = random_cache(B, Hkv, cap, D, 21, view=True)
    dst = cca.kv4_cache(B, Hkv, (keep + 15) // 16 * 16 + 16, D, k_scale=0.5, v_scale=2.0)
    for t in (dst.k_codes, dst.k_scales, dst.v_codes, dst.v_scales):
        t.fill_(0xCD)
    mass = torch.tensor(MASSES[kind](rng, (B, Hkv, cap)), dtype=torch.float32).cuda()
    mo = torch.full((B, Hkv, keep + 5), -7.0, device="cuda")
    dl = i32(lens)
    ws = cca.kv4_workspace(src)
    out, slots = cca.kv4_evict(src, dl, mass, keep, recent, dst, mo, lens_out=dl, ws=ws)       # lengths in place
    assert out is dl and dl.tolist() == [min(n, keep) for n in lens] and cca.attn_status(ws) == 0
    hm = mass.cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(Hkv):
            want = K.evict(hm[b, h], n, keep, recent)
            m = len(want)
            assert slots[b, h].tolist() == want + [-1] * (keep - m)
            idx = torch.tensor(want, dtype=torch.long, device="cuda")
            for a, z in ((src.k_codes, dst.k_codes), (src.k_scales, dst.k_scales), (src.v_codes, dst.v_codes),
                         (src.v_scales, dst.v_scales)):
                assert torch.equal(z[b, h, :m], a[b, h][idx]) and (z[b, h, m:] == 0xCD).all()
            assert torch.equal(mo[b, h, :m].view(torch.int32), mass[b, h][idx].view(torch.int32))
            assert (mo[b, h, m:] == -7).all()


@pytest.mark.parametrize("cap,keep,recent", [(20000, 1000, 17), (20000, 19990, 0), (70000, 4096, 4096), (70000, 5000, 64), (300000, 6000, 5)])
def test_evict_long(cap, keep, recent):
    rng = np.random.default_rng(cap + keep)
    src = random_cache(1, 3, cap, 64, 22)
    dst = cca.kv4_cache(1, 3, (keep + 15) // 16 * 16, 64, k_scale=0.5, v_scale=2.0)
    mass = torch.tensor(np.round(np.exp(2 * rng.normal(size=(1, 3, cap))), 1), dtype=torch.float32).cuda()   # many ties
    out, slots = cca.kv4_evict(src, i32([cap - 3]), mass, keep, recent, dst)
    for h in range(3):
        want = K.evict(mass[0, h].cpu().numpy(), cap - 3, keep, recent)
        assert slots[0, h].tolist() == want
        assert torch.equal(dst.v_codes[0, h, :keep], src.v_codes[0, h][torch.tensor(want, device="cuda")])


def test_evict_reports_bad_lengths():
    src, dst = random_cache(3, 1, 64, 64, 23), cca.kv4_cache(3, 1, 16, 64, k_scale=0.5, v_scale=2.0)
    mass = torch.rand(3, 1, 50, device="cuda")
    ws = cca.kv4_workspace(src)
    out, slots = cca.kv4_evict(src, i32([70, -5, 51]), mass, 16, 2, dst, ws=ws)
    assert cca.attn_status(ws) == 7 and out.tolist() == [16, 0, 16]
    for b in (0, 2):
        assert slots[b, 0].tolist() == K.evict(mass[b, 0].cpu().numpy(), 50, 16, 2)


# ------------------------------------------------------------------ as they are used

def test_prompt_then_decode_then_evict():
    """A prompt runs chunk by chunk (attn_fwd), its keys' weights accumulate, its rows are stored;
    the cache is cut to a budget; tokens are decoded with their rows appended and weights added,
    by a captured graph, and the cache is cut again."""
    rng = np.random.default_rng(41)
    B, H, Hkv, D, L, keep, recent, steps = 2, 8, 2, 128, 500, 128, 32, 24
    q, k, v = 2 * bf16(rng, B, H, L, D), bf16(rng, B, Hkv, L, D), bf16(rng, B, Hkv, L, D)
    chunks = cca.attn_plan(L, 2, cca.PLAN_FLOPS)
    o, lse = cca.forward_streamed(q, k, v, chunks)
    mass = torch.zeros(B, Hkv, L, device="cuda")
    for c in chunks:
        cca.key_mass(q, k, lse, [c], mass_in=mass, mass_out=mass)
    check_mass(q, k, lse, chunks, mass, D ** -0.5)
    full = cca.kv4_cache(B, Hkv, 512, D)
    zero = i32([0] * B)
    cca.kv4_store(full, k, v, zero)
    # the last rows' attention over the cache is the prompt's own, up to the 4-bit keys and values
    o4, lse4 = cca.kv4_attention(q[:, :, L - 4:], full, i32([L] * B))
    check_attend(q[:, :, L - 4:], full, [L] * B, o4, lse4)
    small, spare = (cca.kv4_cache(B, Hkv, 160, D) for _ in range(2))
    m1, m2 = torch.zeros(B, Hkv, 160, device="cuda"), torch.zeros(B, Hkv, 160, device="cuda")
    lens, slots = cca.kv4_evict(full, i32([L] * B), mass, keep, recent, small, m1)
    for b in range(B):
        for h in range(Hkv):
            assert slots[b, h].tolist() == K.evict(mass[b, h].cpu().numpy(), L, keep, recent)
    # decoding: one graph, its inputs copied in
    nq, nk, nv = (torch.zeros(B, x, 1, D, dtype=torch.bfloat16, device="cuda") for x in (H, Hkv, Hkv))
    ws = cca.kv4_workspace(small, nq, mass=True)

    def step():
        cca.kv4_store(small, nk, nv, lens, ws=ws)
        lens.add_(1)
        return cca.kv4_attention(nq, small, lens, mass_in=m1, mass_out=m1, ws=ws)

    state = [t.clone() for t in (lens, m1, small.k_codes, small.k_scales, small.v_codes, small.v_scales)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, glse = step()
    for t, s in zip((lens, m1, small.k_codes, small.k_scales, small.v_codes, small.v_scales), state):
        t.copy_(s)
    for i in range(steps):
        before = m1.clone()
        nq.copy_(2 * bf16(rng, B, H, 1, D)), nk.copy_(bf16(rng, B, Hkv, 1, D)), nv.copy_(bf16(rng, B, Hkv, 1, D))
        graph.replay()
        n = [keep + i + 1] * B
        assert lens.tolist() == n
        check_attend(nq, small, n, go, glse, None, before, m1, kept_tail=0.0)
    lens2, slots = cca.kv4_evict(small, lens, m1, keep, recent, spare, m2, ws=ws)
    assert cca.attn_status(ws) == 0 and lens2.tolist() == [keep] * B
    for b in range(B):
        for h in range(Hkv):
            assert slots[b, h].tolist() == K.evict(m1[b, h].cpu().numpy(), keep + steps, keep, recent)


def test_chunk_over_a_stored_context():
    """A further chunk of a prompt attends (attn_fwd) to a context that is read back from the cache."""
    rng = np.random.default_rng(43)
    H, D, L, new = 4, 64, 300, 100
    k, v = bf16(rng, 1, H, L, D), bf16(rng, 1, H, L, D)
    c = cca.kv4_cache(1, H, 304, D)
    cca.kv4_store(c, k, v, i32([0]))
    kk, vv = cca.kv4_load(c, i32([0]), L)
    q = 2 * bf16(rng, 1, H, L, D)
    o, lse = cca.forward(q, kk, vv, [(L - new, L, 0, 0)])
    o4, lse4 = cca.kv4_attention(q[:, :, L - new:], c, i32([L]))
    check_attend(q[:, :, L - new:], c, [L], o4, lse4)
    assert (o[:, :, L - new:].double() - o4.double()).abs().max() <= 2e-2
    assert (lse[:, :, L - new:] - lse4).abs().max() <= 1e-3


def test_calls_on_two_streams_and_wrong_sizes():
    rng = np.random.default_rng(45)
    c = random_cache(2, 2, 2048, 128, 46)
    q = [bf16(rng, 2, 8, 1, 128) for _ in range(2)]
    want = [cca.kv4_attention(x, c, i32([2048, 700])) for x in q]
    ws = [cca.kv4_workspace(c, q[0]) for _ in range(2)]
    lens = i32([2048, 700])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for x, w, s in zip(q, ws, streams):
            with torch.cuda.stream(s):
                got.append(cca.kv4_attention(x, c, lens, ws=w))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])
    for bad in (lambda: cca.kv4_attention(q[0][:1], c, lens), lambda: cca.kv4_attention(q[0], c, lens[:1]),
                lambda: cca.kv4_attention(q[0], c, lens.long()), lambda: cca.kv4_attention(q[0].half(), c, lens),
                lambda: cca.kv4_attention(q[0][:, :3], c, lens), lambda: cca.kv4_attention(q[0], c, lens, mass_in=torch.zeros(2, 2, 2048, device="cuda")),
                lambda: cca.kv4_attention(q[0], c, lens, mass_out=torch.zeros(2, 3, 2048, device="cuda")),
                lambda: cca.kv4_store(c, q[0][:, :2], q[1][:, :2, :, :64], lens),
                lambda: cca.kv4_evict(c, lens, torch.zeros(2, 2, 2048, device="cuda"), 16, 2, c)):
        with pytest.raises(cca.AttnError):
            bad()


@pytest.mark.parametrize("raw", [False, True])
def test_a_given_stream_holds_what_a_call_allocates(raw, monkeypatch):
    """With stream= alone, workspaces and outputs are allocated (and zeroed, and given back) on that stream."""
    rng = np.random.default_rng(47)
    c, d = random_cache(2, 2, 1024, 64, 48), cca.kv4_cache(2, 2, 256, 64, k_scale=0.5, v_scale=2.0)
    q, lens = bf16(rng, 2, 4, 1, 64), i32([1000, 30])
    mass = torch.rand(2, 2, 1024, device="cuda")
    p, rows, zero = bf16(rng, 2, 4, 300, 64), bf16(rng, 2, 2, 9, 64), i32([0, 16])
    chunks = [(0, 300, 0, 0)]
    _, p_lse = cca.forward(p, p, p, chunks)
    side = torch.cuda.Stream()
    seen = []

    def watched(f):
        def g(*a, **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return f(*a, **kw)
        return g

    def calls(**kw):
        cca.kv4_store(c, rows, rows, zero, **kw)
        k, v = cca.kv4_load(c, zero, 9, **kw)
        o, lse = cca.kv4_attention(q, c, lens, **kw)
        n, slots = cca.kv4_evict(c, lens, mass, 200, 8, d, **kw)
        return k, v, o, lse, n, slots, cca.key_mass(p, p, p_lse, chunks, **kw)

    want = calls()
    torch.cuda.synchronize()
    monkeypatch.setattr(cca.kv4, "kv4_workspace", watched(cca.kv4.kv4_workspace))
    monkeypatch.setattr(cca, "workspace", watched(cca.workspace))
    here = torch.cuda.current_stream().cuda_stream
    got = calls(stream=side.cuda_stream if raw else side)
    assert torch.cuda.current_stream().cuda_stream == here
    torch.cuda.synchronize()
    assert seen == [side.cuda_stream] * 5
    for x, y in zip(got, want):
        assert torch.equal(x, y)
