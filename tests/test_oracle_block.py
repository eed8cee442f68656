"""CPU pins of the block attention and sampling oracles, and the refusals of
the three block_* calls beside the acceptance (checked on the host, before
anything touches a device)."""
import math

import numpy as np
import pytest

from mxfp4_moe_block_b200 import _lib, build
from oracle import attention as oatt
from oracle import sample as osam


# ------------------------------------------------------------------ oracles --

def test_rotation_is_a_turn():
    """Norm kept, angles add up, and scores depend on the distance alone."""
    rng = np.random.default_rng(1)
    for inter in (False, True):
        x, y = rng.standard_normal(8), rng.standard_normal(8)
        f = np.array([1.0, 0.3, 0.01])
        cs = lambda p: np.concatenate([np.cos(p * f), np.sin(p * f)])
        r = lambda v, p: oatt.rotate(v, cs(p), inter)
        assert math.isclose(np.linalg.norm(r(x, 7)), np.linalg.norm(x))
        assert np.allclose(r(r(x, 3), 4), r(x, 7))
        assert np.allclose(r(x, 9) @ r(y, 5), r(x, 104) @ r(y, 100))
        assert np.array_equal(r(x, 7)[6:], x[6:])
    # by hand: a quarter turn takes (1, 0) to (0, 1), halves and neighbours
    q = np.array([0.0, 0.0, 1.0, 1.0])
    assert np.array_equal(oatt.rotate(np.array([1.0, 2.0, 3.0, 4.0]), q, False), [-3, -4, 1, 2])
    assert np.array_equal(oatt.rotate(np.array([1.0, 2.0, 3.0, 4.0]), q, True), [-2, 1, -4, 3])


def test_append_places_and_skips():
    k = np.full((3, 1, 2, 2), 9.0)
    v, q = k.copy(), np.full((3, 2, 1, 2), 7.0)
    qkv = np.arange(3 * 2 * 3 * 2, dtype=np.float64).reshape(3, 2, 3, 2) + 1
    # slot 0 idle; slot 1 has one position only; slot 2 ends at position 3
    bad = oatt.kv_append(qkv, [0, 1, 4], np.array([[0, 0], [2, 0], [1, 0]]), k, v, q, norm=False)
    assert not bad
    assert (q[0] == 7).all() and (q[1, 0] == 7).all() and np.array_equal(q[1, 1], qkv[1, 1, :1])
    assert np.array_equal(k[2, 0, 0], qkv[1, 1, 1]) and (k[2, 0, 1] == 9).all()
    assert np.array_equal(k[0, 0], qkv[2, :, 1]) and np.array_equal(v[0, 0], qkv[2, :, 2])
    assert (k[1] == 9).all()
    for kv_len, table in (([5], [[0, 0]]), ([4], [[0, 3]]), ([4], [[0, -1]])):
        assert oatt.kv_append(qkv[:1], kv_len, np.array(table), k, v, q[:1], norm=False)


def test_attention_by_hand():
    """Uniform scores give means; a window, an empty slot, a negative position
    and a bad page each leave out what they should."""
    k = np.zeros((3, 1, 2, 4))
    v = np.arange(3 * 2 * 4, dtype=np.float64).reshape(3, 1, 2, 4)
    q = np.ones((1, 2, 2, 4))
    t = np.array([[2, 0]])
    flat = np.concatenate([v[2, 0], v[0, 0]])
    out, _, bad = oatt.attention(q, k, v, t, [3])
    assert not bad and np.allclose(out[0, 0], flat[:2].mean(0)) and np.allclose(out[0, 1], flat[:3].mean(0))
    out, _, _ = oatt.attention(q, k, v, t, [4], window=1)
    assert np.allclose(out[0, :, 0], flat[2:4])
    out, _, _ = oatt.attention(q, k, v, t, [1])
    assert (out[0, 0] == 0).all() and np.allclose(out[0, 1], flat[0])
    assert (oatt.attention(q, k, v, t, [0])[0] == 0).all()
    out, _, bad = oatt.attention(q, k, v, np.array([[2, 3]]), [4])
    assert bad and np.allclose(out[0, 1], flat[:2].mean(0))
    out, _, bad = oatt.attention(q, k, v, t, [5])
    assert bad and (out == 0).all()


def test_attention_is_softmax():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((4, 2, 3, 8)), rng.standard_normal((4, 2, 3, 8))
    q = rng.standard_normal((1, 1, 4, 8))
    out, _, _ = oatt.attention(q, k, v, np.array([[3, 1, 0, 2]]), [10], scale=0.7)
    j = np.arange(10)
    page = np.array([3, 1, 0, 2])[j // 3]
    z = 0.7 * k[page, 1, j % 3] @ q[0, 0, 2]
    assert np.allclose(out[0, 0, 2], (np.exp(z)[:, None] * v[page, 1, j % 3]).sum(0) / np.exp(z).sum())


def test_filters_by_hand():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.2, 0.1]))
    kept = lambda **f: osam.kept_tokens(l, **f)[0]
    assert kept() == [1, 2, 3, 0, 4]                       # ties to the lowest index
    assert kept(top_k=2) == [1, 2] and kept(top_k=9) == kept(top_k=0) == kept()
    assert kept(top_p=0.3) == [1] and kept(top_p=0.0) == [1] and kept(top_p=-1.0) == [1]
    assert kept(top_p=0.59) == [1, 2] and kept(top_p=0.61) == [1, 2, 3]
    assert kept(min_p=0.4) == [1, 2, 3] and kept(min_p=0.9) == [1] and kept(min_p=3.0) == [1]
    assert kept(top_k=3, top_p=0.7) == [1, 2]              # of the top 3's mass 0.8: 0.56
    assert kept(temperature=0.0) == kept(temperature=-1.0) == kept(temperature=float("nan")) == [1]
    assert kept(temperature=0.5, top_p=0.8) == [1, 2, 3]   # weights 16 4 4 1 1 of 26: 20.8 wanted
    _, p = osam.sample_row(l, top_k=2)
    assert np.allclose(p, [0, 2 / 3, 1 / 3, 0, 0])


def test_draw_borders():
    """Equal masses: token v is drawn for u in [v/4, (v+1)/4), exactly."""
    l = np.zeros(4)
    step = 2.0 ** -24
    for v in range(4):
        assert osam.sample_row(l, v / 4)[0] == v
        assert osam.sample_row(l, (v + 1) / 4 - step)[0] == v
    masked = np.array([-np.inf, 0.0, np.nan, 0.0])
    assert osam.sample_row(masked, 0.0)[0] == 1 and osam.sample_row(masked, 0.5)[0] == 3
    t, p = osam.sample_row(np.array([-np.inf, np.nan]), 0.5)
    assert t == -1 and (p == 0).all()
    t, p = osam.sample_row(np.array([0.0, np.inf]), 0.5)
    assert t == 1 and np.array_equal(p, [0, 1])


# ----------------------------------------------------------------- refusals --

@pytest.fixture(scope="module")
def library():
    build.build()
    return _lib.lib()


A = 4096     # a dummy address, 256-byte aligned; every refusal comes before its use


def append(L, **kw):
    a = dict(qkv=A, S=1, N=1, Hq=8, Hkv=2, D=128, norm=1, qw=None, kw=None, eps=1e-6, cs=A,
             max_pos=16, rot=64, inter=0, kv_len=A, table=A, max_pages=4, k=A, v=A, pages=4, ps=16,
             q_out=A, stream=None)
    a.update(kw)
    return L.block_kv_append(*a.values())


def attention(L, **kw):
    a = dict(q=A, S=1, N=1, Hq=8, Hkv=2, D=128, k=A, v=A, pages=4, ps=16, table=A, max_pages=4,
             kv_len=A, scale=1.0, window=0, out=A, ws=A, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return L.block_attention(*a.values())


def sample(L, **kw):
    a = dict(logits=A, S=1, K=1, V=16, t=None, k=None, p=None, m=None, u=A, token=A, probs=None,
             stream=None)
    a.update(kw)
    return L.block_sample(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(N=0), 1), (dict(Hkv=0), 1), (dict(Hq=7), 1), (dict(Hq=0), 1),
    (dict(D=96), 2), (dict(D=0), 1), (dict(N=65), 2), (dict(Hq=2048), 2),
    (dict(S=(1 << 20) + 1), 2), (dict(rot=24), 1), (dict(rot=144), 1), (dict(rot=-16), 1),
    (dict(cs=None), 1), (dict(max_pos=0), 1), (dict(max_pages=0), 1), (dict(pages=0), 1),
    (dict(ps=0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(max_pages=1 << 20, ps=1 << 12), 2), (dict(qkv=None), 1), (dict(kv_len=None), 1),
    (dict(table=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(q_out=None), 1),
    (dict(qkv=A + 2), 1), (dict(k=A + 8), 1), (dict(v=A + 2), 1), (dict(q_out=A + 4), 1),
    (dict(cs=A + 4), 1), (dict(qw=A + 2), 1), (dict(kw=A + 2), 1), (dict(S=0, qkv=None), 0),
    (dict(max_pages=(1 << 18) + 1, ps=1 << 12), 2), (dict(max_pages=1 << 18, ps=1 << 12, qkv=None), 1)])
def test_append_refusals(library, kw, status):
    assert append(library, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(N=0), 1), (dict(N=65), 2), (dict(Hq=7), 1), (dict(D=80), 2),
    (dict(pages=0), 1), (dict(ps=0), 1), (dict(max_pages=0), 1), (dict(window=-1), 1),
    (dict(scale=float("inf")), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(max_pages=1 << 20, ps=1 << 12), 2), (dict(q=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(table=None), 1), (dict(kv_len=None), 1), (dict(out=None), 1),
    (dict(ws=None), 1), (dict(ws_bytes=16), 4), (dict(ws=A + 16), 4), (dict(q=A + 2), 1),
    (dict(k=A + 8), 1), (dict(v=A + 8), 1), (dict(out=A + 2), 1), (dict(S=0, q=None), 0),
    (dict(max_pages=(1 << 18) + 1, ps=1 << 12), 2), (dict(max_pages=1 << 18, ps=1 << 12, q=None), 1)])
def test_attention_refusals(library, kw, status):
    assert attention(library, **kw) == status


def test_attention_workspace_query(library):
    assert library.block_attention_workspace_bytes(4, 8, 64, 8, 128) > 0
    assert library.block_attention_workspace_bytes(4, 8, 64, 7, 128) == 0
    assert library.block_attention_workspace_bytes(4, 8, 64, 8, 100) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(K=0), 1), (dict(V=0), 1), (dict(V=393217), 2), (dict(K=65), 2),
    (dict(S=1 << 15, K=64), 2), (dict(u=None), 1), (dict(token=None), 1),
    (dict(u=None, token=None), 1), (dict(logits=None), 1), (dict(S=0, logits=None), 0)])
def test_sample_refusals(library, kw, status):
    assert sample(library, **kw) == status


def test_binding_wants_cuda_tensors():
    import torch

    import mxfp4_moe_block_b200 as mm
    with pytest.raises(ValueError, match="CUDA"):
        mm.block_sample(torch.zeros(1, 1, 8))
