"""GPU parity of the block's cache append, attention and sampling against the
oracle (float64) on small shapes, and a run of all of them as one verify step.

Tolerances (HALF = half a bf16 step, 2^-8 of a value; EPS = half a float
step, 2^-24):
* append: one rounding to bf16 of a value computed in float.  The norm sums
  D <= 256 squares by a tree of at most 8 + 8 additions and takes a root, a
  quotient and two products: relative error below 32 EPS; the rotation adds
  two such products, each off by at most 2 EPS more.  In all HALF of the value
  plus 2^-18 of |a| + |b|, the pair's magnitudes.
* attention: a score z = scale q.k is off by at most (D + 4) EPS scale |q|.|k|
  =: dz, its weight relatively by 2 dz + 2^-20 (exponential and its argument),
  the weight's rounding to bf16 adds HALF; numerator and sum carry these, so
  the result is off by (HALF + 4 dz + 2^-17) of the weighted mean of |v|, and by
  HALF of itself for the last rounding.
* sampling: tokens equal; a probability is a weight times the reciprocal of a
  sum (both within 2^-44 as doubles), three roundings to float: 3 EPS < 2^-22
  relative, or one float denormal.
"""
import math

import numpy as np
import pytest
import torch

import mxfp4_moe_block_b200 as mm
from oracle import accept as oacc
from oracle import attention as oatt
from oracle import sample as osam

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = torch.finfo(torch.bfloat16).eps / 2
EPS = torch.finfo(torch.float32).eps / 2
BAD_INDEX, NO_MASS = (5, 5), (5, 2)


@pytest.fixture(autouse=True)
def clean_status():
    mm.moe_clear_device_status()
    yield
    mm.moe_clear_device_status()


def bf16(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32)


def tables(kv_len, page, pages, seed, spare=1):
    """Scattered pages; entries past a sequence's end hold ids no pool has."""
    g = np.random.default_rng(seed)
    need = [-(-max(int(n), 0) // page) for n in kv_len]
    ids = g.permutation(pages)
    assert sum(need) <= pages
    t = np.full((len(kv_len), max(need) + spare), -7, np.int32)
    at = 0
    for s, m in enumerate(need):
        t[s, :m] = ids[at:at + m]
        at += m
    return t


def cos_sin(max_pos, rot, base=1e4):
    a = np.arange(max_pos)[:, None] * base ** (-np.arange(rot // 2) / max(rot // 2, 1))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float()


# ------------------------------------------------------------------- append --

APPEND = [
    # S, N, Hq, Hkv, D, rot, page, lens, norm, weights, interleaved
    (1, 1, 8, 1, 128, 128, 16, [1], True, True, False),
    (3, 5, 6, 2, 128, 64, 24, [5, 0, 100], True, True, True),
    (4, 8, 7, 7, 64, 64, 1, [8, 9, 3, 17], False, False, False),
    (2, 33, 40, 8, 256, 256, 32, [33, 500], True, False, False),
    (2, 64, 3, 3, 64, 16, 100, [64, 321], True, True, True),
    (5, 2, 2, 1, 256, 0, 8, [2, 7, 8, 9, 1], True, True, False),
    (2, 3, 12, 2, 128, 32, 7, [3, -4], False, False, True),
    (9, 4, 64, 8, 128, 96, 16, [4, 5, 15, 16, 17, 18, 19, 20, 21], True, True, False),
]


def append_case(c, seed):
    S, N, Hq, Hkv, D, rot, page, lens, norm, weights, inter = c
    pages = sum(-(-max(n, 0) // page) for n in lens) + 3
    st = dict(qkv=bf16((S, N, Hq + 2 * Hkv, D), seed, 2.0), kv_len=i32(lens),
              block_table=i32(tables(lens, page, pages, seed)),
              k_cache=bf16((pages, Hkv, page, D), seed + 1), v_cache=bf16((pages, Hkv, page, D), seed + 2),
              q_out=bf16((S, N, Hq, D), seed + 3), cos_sin=cos_sin(max(lens) + 2, rot) if rot else None,
              q_weight=bf16((D,), seed + 4) if weights else None,
              k_weight=bf16((D,), seed + 5) if weights else None)
    return st, dict(norm=norm, eps=1e-5, interleaved=inter)


def check_append(st, opt, run=None):
    """Runs the call on copies and compares every value of q_out and the caches."""
    ref = {k: None if v is None else f64(v) for k, v in st.items()}
    old = {k: ref[k].copy() for k in ("q_out", "k_cache", "v_cache")}
    bad = oatt.kv_append(**{**ref, "kv_len": st["kv_len"].numpy(),
                            "block_table": st["block_table"].numpy()}, **opt)
    dev = {k: None if v is None else v.to(DEV) for k, v in st.items()}
    (run or (lambda: mm.block_kv_append(**dev, **opt)))()
    # the magnitudes a rotation mixes, by the same path without the signs
    mag = {k: v.copy() for k, v in old.items()}
    a = dict(ref, q_weight=None if ref["q_weight"] is None else abs(ref["q_weight"]),
             k_weight=None if ref["k_weight"] is None else abs(ref["k_weight"]))
    rot = 0 if ref["cos_sin"] is None else ref["cos_sin"].shape[1]
    if rot:            # |a| + |b| for both of a pair: turn (|a|, |b|) by cos = 1, sin = -1, then +1
        ones = np.concatenate([np.ones(rot // 2), -np.ones(rot // 2)])
        parts = []
        for sign in (1, -1):
            m = {k: v.copy() for k, v in old.items()}
            cs = np.tile(np.concatenate([ones[:rot // 2], sign * ones[rot // 2:]]), (len(ref["cos_sin"]), 1))
            oatt.kv_append(**{**a, **m, "qkv": abs(ref["qkv"]), "cos_sin": cs,
                              "kv_len": st["kv_len"].numpy(), "block_table": st["block_table"].numpy()}, **opt)
            parts.append(m)
        mag = {k: np.maximum(abs(parts[0][k]), abs(parts[1][k])) for k in mag}
    else:
        mag = {k: abs(ref[k]) for k in mag}
    for k in ("q_out", "k_cache"):
        got, want = f64(dev[k]), ref[k]
        same = want == old[k]
        assert np.array_equal(got[same], want[same]), f"{k}: rows that should stay changed"
        lim = HALF * abs(want) + 2.0 ** -18 * mag[k]
        assert (abs(got - want) <= lim).all(), (k, float((abs(got - want) - lim).max()))
    assert np.array_equal(f64(dev["v_cache"]), ref["v_cache"])
    assert mm.moe_get_device_status() == (BAD_INDEX if bad else (0, 0))
    return dev


@pytest.mark.parametrize("c", APPEND, ids=str)
def test_append(c):
    st, opt = append_case(c, 11)
    check_append(st, opt)


def test_append_wide_and_many_tokens():
    """More than one group of heads a token, hundreds of tokens."""
    st, opt = append_case((40, 16, 64, 8, 64, 64, 16, [16 + 3 * s for s in range(40)], True, True, False), 5)
    check_append(st, opt)


def test_append_allocates_zeroed_queries():
    st, opt = append_case(APPEND[1], 3)
    st["q_out"] = None
    q = mm.block_kv_append(**{k: None if v is None else v.to(DEV) for k, v in st.items()}, **opt)
    assert (q[1] == 0).all() and (q[0] != 0).any()


@pytest.mark.parametrize("what", ["page", "negative", "table", "cos_sin"])
def test_append_leaves_out_bad_places(what):
    """One sequence's token has no place: it is reported and left out, the
    other sequence's tokens are not touched by it."""
    st, opt = append_case((2, 4, 4, 2, 128, 128, 8, [12, 30], True, True, False), 21)
    if what == "page":
        st["block_table"][0, 1] = st["k_cache"].shape[0]
    elif what == "negative":
        st["block_table"][0, 1] = -1
    elif what == "table":
        st["block_table"] = st["block_table"][:, :3].contiguous()
    else:
        st["cos_sin"] = st["cos_sin"][:28].contiguous()
    check_append(st, opt)


# ---------------------------------------------------------------- attention --

ATTENTION = [
    # S, N, Hq, Hkv, D, page, lens, window
    (1, 1, 8, 1, 128, 16, [1], 0),
    (1, 1, 64, 8, 128, 16, [777], 0),
    (3, 8, 8, 2, 128, 24, [300, 0, 5], 0),
    (4, 1, 4, 4, 64, 1, [1, 127, 128, 129], 0),
    (2, 16, 16, 2, 64, 32, [16, 1000], 0),
    (2, 33, 14, 2, 128, 64, [33, 260], 0),
    (1, 64, 64, 1, 64, 16, [70], 0),
    (2, 5, 6, 2, 256, 16, [64, 195], 0),
    (1, 20, 8, 1, 256, 100, [333], 0),
    (3, 8, 8, 4, 64, 16, [900, 7, 128], 128),
    (2, 3, 4, 2, 128, 8, [255, 400], 1),
    (2, 16, 8, 1, 128, 128, [512, 513], 20),
    (1, 4, 4, 2, 256, 3, [131], 64),
    (7, 2, 2, 1, 128, 16, [2, 15, 16, 17, -3, 31, 1], 0),
    (1, 1, 16, 16, 128, 16, [4097], 0),
]


def attention_case(c, seed, q_scale=2.0):
    S, N, Hq, Hkv, D, page, lens, window = c
    pages = sum(-(-max(n, 0) // page) for n in lens) + 3
    st = dict(q=bf16((S, N, Hq, D), seed, q_scale), k_cache=bf16((pages, Hkv, page, D), seed + 1),
              v_cache=bf16((pages, Hkv, page, D), seed + 2),
              block_table=i32(tables(lens, page, pages, seed)), kv_len=i32(lens))
    # what no token sees holds NaN: pages not in a table, rows at or past the end
    seen = np.zeros((pages, page), bool)
    for s, n in enumerate(lens):
        for j in range(max(0, n - N - window + 1) if window else 0, max(n, 0)):
            seen[st["block_table"][s, j // page], j % page] = True
    for k in ("k_cache", "v_cache"):
        st[k].permute(0, 2, 1, 3)[torch.from_numpy(~seen)] = float("nan")
    return st, window


def check_attention(st, window, got, scale=None, status=(0, 0)):
    want, spread, bad = oatt.attention(f64(st["q"]), f64(st["k_cache"]), f64(st["v_cache"]),
                                       st["block_table"].numpy(), st["kv_len"].numpy(), scale, window)
    assert mm.moe_get_device_status() == (BAD_INDEX if bad else (0, 0))
    D = st["q"].shape[-1]
    k = np.nan_to_num(f64(st["k_cache"]))
    big = np.linalg.norm(f64(st["q"]), axis=-1).max() * np.linalg.norm(k, axis=-1).max()
    dz = (D + 4) * EPS * (D ** -0.5 if scale is None else abs(scale)) * big
    lim = HALF * abs(want) + (HALF + 4 * dz + 2.0 ** -17) * spread
    got = f64(got)
    assert np.isfinite(got).all()
    over = abs(got - want) - lim
    assert (over <= 0).all(), (float(over.max()), np.unravel_index(over.argmax(), over.shape))


def to_dev(st):
    return {k: v.to(DEV) for k, v in st.items()}


@pytest.mark.parametrize("c", ATTENTION, ids=str)
def test_attention(c):
    st, window = attention_case(c, 31)
    out = torch.full(st["q"].shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    mm.block_attention(**to_dev(st), window=window, out=out)
    check_attention(st, window, out)


@pytest.mark.parametrize("D,lens", [(64, [2000, 3, 700]), (128, [3000, 130, 1]), (256, [900, 64, 65])])
def test_attention_many_splits_and_ragged_lengths(D, lens):
    """Long sequences beside short ones: pieces of one sequence on many CTAs,
    many sequences on one."""
    c = (40, 4, 4, 2, D, 16, (lens * 14)[:40], 0)
    st, window = attention_case(c, 77)
    check_attention(st, window, mm.block_attention(**to_dev(st)))


@pytest.mark.parametrize("scale", [0.0, 0.02, 3.0])
def test_attention_scales(scale):
    """Scores from all equal to one key taking everything;
    growing scores make every tile raise the running maximum."""
    c = (2, 4, 8, 2, 128, 16, [600, 150], 0)
    st, window = attention_case(c, 41, 1.0)
    ramp = torch.linspace(0.2, 3.0, 600)
    for s, n in enumerate(c[6]):
        for j in range(n):
            st["k_cache"][st["block_table"][s, j // 16], :, j % 16] *= ramp[j]
    check_attention(st, window, mm.block_attention(**to_dev(st), scale=scale), scale)


def test_attention_extreme_scores():
    """Scores of +-3e4 (weights that underflow to 0 beside a weight of 1)."""
    st, window = attention_case((1, 2, 4, 2, 128, 16, [300], 0), 43)
    st["q"].zero_()
    st["q"][..., 0] = 256.0
    k = st["k_cache"].permute(0, 2, 1, 3)
    k[...] = torch.where(torch.isnan(k), k, torch.zeros_like(k))
    for j in range(300):
        st["k_cache"][st["block_table"][0, j // 16], :, j % 16, 0] = 128.0 * (-1) ** j * (1 + (j % 7 == 3))
    check_attention(st, window, mm.block_attention(**to_dev(st), scale=1.0), 1.0)


@pytest.mark.parametrize("what", ["page", "negative", "table"])
def test_attention_leaves_out_bad_pages(what):
    st, window = attention_case((3, 2, 4, 2, 64, 16, [100, 200, 40], 0), 51)
    for k in ("k_cache", "v_cache"):
        st[k] = torch.nan_to_num(st[k])
    if what == "page":
        st["block_table"][1, 3] = st["k_cache"].shape[0]
    elif what == "negative":
        st["block_table"][1, 0] = -1
    else:
        st["kv_len"][1] = 16 * st["block_table"].shape[1] + 1
    check_attention(st, window, mm.block_attention(**to_dev(st)))
    # the next call is green again
    mm.moe_clear_device_status()
    st, window = attention_case(ATTENTION[2], 52)
    check_attention(st, window, mm.block_attention(**to_dev(st)))


def test_attention_pages_before_the_window_are_not_used():
    """Pages that slid out of the window may have been given away: their table
    entries hold anything."""
    st, window = attention_case((2, 4, 4, 2, 128, 16, [500, 333], 64), 61)
    for s, n in enumerate([500, 333]):
        st["block_table"][s, : (n - 4 - 64 + 1) // 16] = 10 ** 9
    check_attention(st, window, mm.block_attention(**to_dev(st), window=window))


@pytest.mark.parametrize("c", [
    (3, 8, 8, 4, 64, 16, [900, 7, 128], 100), (2, 8, 16, 2, 128, 16, [600, 1030], 0),
    (2, 16, 16, 2, 128, 24, [400, 1500], 200), (2, 33, 14, 2, 128, 64, [33, 260], 40),
    (4, 5, 6, 2, 256, 16, [64, 195, 1000, 6], 70), (1, 64, 32, 1, 64, 128, [500], 65)], ids=str)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_attention_values_that_are_not_finite_reach_no_other_token(c, value):
    """The last token's value, and that of the first key in the window: of the
    block's tokens only the last, only the first, sees it."""
    S, N, Hq, Hkv, D, page, lens, window = c
    st, _ = attention_case(c, 65)
    d = to_dev(st)
    for s, n in enumerate(lens):
        marks = [n - 1] + ([n - N - window + 1] if window and n - N - window >= 0 else [])
        for j in marks:
            d["v_cache"][st["block_table"][s, j // page], :, j % page, 5:D:7] = value
    out = mm.block_attention(**d, window=window)
    for s, n in enumerate(lens):
        seeing = [N - 1] + ([0] if window and n - N - window >= 0 else [])
        for i in seeing:
            assert not torch.isfinite(out[s, i, :, 5]).any()
            assert torch.isfinite(out[s, i, :, 4]).all()
            # (their other dims hold what the oracle has; these are set to it)
            want = oatt.attention(f64(st["q"])[s:s + 1], f64(st["k_cache"]), f64(st["v_cache"]),
                                  st["block_table"].numpy()[s:s + 1], st["kv_len"].numpy()[s:s + 1],
                                  None, window)[0]
            out[s, i, :, 5:D:7] = torch.from_numpy(want[0, i, :, 5:D:7]).to(out)
    check_attention(st, window, out)


def test_attention_shared_pages():
    """Two sequences share a prefix's pages."""
    st, window = attention_case((2, 2, 8, 2, 128, 16, [90, 90], 0), 63)
    st["block_table"][1, :4] = st["block_table"][0, :4]
    check_attention(st, window, mm.block_attention(**to_dev(st)))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [40, 48, 200, 256, 384, 512])
def test_attention_page_sizes(D, page):
    """Pages smaller and larger than a tile, multiples of it and not, whole and
    seen in part at both ends."""
    for window in (0, 300):
        st, window = attention_case((3, 3, 6, 2, D, page, [1500, 511, 2 * page + 1], window), page + window)
        check_attention(st, window, mm.block_attention(**to_dev(st), window=window))


def test_attention_many_rows_and_splits():
    """512 rows to a key/value head (four blocks of rows), cut among the GPU."""
    st, window = attention_case((2, 64, 16, 2, 64, 16, [2000, 300], 0), 67)
    check_attention(st, window, mm.block_attention(**to_dev(st)))


@pytest.mark.parametrize("D,page", [(64, 16), (128, 48), (128, 5), (256, 64)])
def test_attention_bad_pages_in_the_window(D, page):
    st, window = attention_case((4, 6, 4, 2, D, page, [700, 90, 300, 1000], 250), 69)
    for k in ("k_cache", "v_cache"):
        st[k] = torch.nan_to_num(st[k])
    for s, n in enumerate([700, 90, 300, 1000]):
        st["block_table"][s, (n - 1) // page - s] = st["k_cache"].shape[0] + s
        st["block_table"][s, max(0, n - 200) // page] = -1
    check_attention(st, window, mm.block_attention(**to_dev(st), window=window))


@pytest.mark.parametrize("page,D", [(1 << 16, 64), (1 << 14, 256), (24, 128)])
def test_attention_positions_near_the_limit(page, D):
    """Lengths just below 2^30 behind a window, and a window past every position."""
    pages = (1 << 30) // page
    N, window, n = 9, 130, pages * page - 3
    g = torch.Generator().manual_seed(70)
    st = dict(q=bf16((2, N, 4, D), 1, 2.0), k_cache=bf16((4, 2, page, D), 2),
              v_cache=bf16((4, 2, page, D), 3), kv_len=i32([n, 5]),
              block_table=torch.randint(0, 4, (2, pages), generator=g, dtype=torch.int32))
    check_attention(st, window, mm.block_attention(**to_dev(st), window=window))
    st["kv_len"] = i32([70, 5])
    for big in ((1 << 31) - 1, 1 << 30):
        check_attention(st, big, mm.block_attention(**to_dev(st), window=big))


@pytest.mark.parametrize("page", [16, 24])
def test_cache_offsets_past_32_bits(page):
    """Pages at the far end of caches of more than 2^32 elements: append, then
    attend."""
    S, N, Hq, Hkv, D, n = 2, 4, 8, 8, 128, 300
    pages = (1 << 32) // (Hkv * page * D) + 60
    kc, vc = (torch.empty((pages, Hkv, page, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    need = -(-n // page)
    table = pages - 1 - torch.arange(S * need, dtype=torch.int32).reshape(S, need)
    first = pages - S * need
    for t, seed in ((kc, 5), (vc, 6)):
        t[first:] = bf16((S * need, Hkv, page, D), seed).to(DEV)
    qkv, kv_len = bf16((S, N, Hq + 2 * Hkv, D), 7), i32([n, n - 1])
    q = mm.block_kv_append(qkv.to(DEV), kv_len.to(DEV), table.to(DEV), kc, vc, norm=False)
    out = mm.block_attention(q, kc, vc, table.to(DEV), kv_len.to(DEV))
    st = dict(q=qkv[:, :, :Hq], k_cache=kc[first:].cpu(), v_cache=vc[first:].cpu(),
              block_table=table - first, kv_len=kv_len)
    assert torch.equal(q.cpu(), st["q"])
    for s in range(S):
        for i in range(N):
            p = int(kv_len[s]) - N + i
            row = st["k_cache"][st["block_table"][s, p // page], :, p % page]
            assert torch.equal(row, qkv[s, i, Hq:Hq + Hkv])
    check_attention(st, 0, out)


def test_attention_two_calls_at_once():
    """Two streams, a workspace each, many calls in flight."""
    cases = [attention_case((6, 8, 16, 2, 128, 16, [1500, 20, 900, 0, 8, 400], 0), 72)[0],
             attention_case((3, 3, 8, 4, 64, 24, [700, 2000, 33], 0), 73)[0]]
    dev = [to_dev(c) for c in cases]
    outs = [[torch.empty_like(d["q"]) for _ in range(6)] for d in dev]
    streams = [torch.cuda.Stream() for _ in dev]
    ws = [mm.alloc_attention_workspace(*d["q"].shape[:3], d["k_cache"].shape[1], d["q"].shape[3], DEV) for d in dev]
    torch.cuda.synchronize()
    for i in range(6):
        for d, o, st, w in zip(dev, outs, streams, ws):
            mm.block_attention(**d, out=o[i], workspace=w, stream=st)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        check_attention(c, 0, o[0])
        assert all(torch.equal(o[0], x) for x in o[1:])


@pytest.mark.parametrize("c", [(40, 2, 16, 8, 128, 16, [600, 250], 0), (40, 8, 48, 8, 128, 16, [600, 250], 0),
                               (40, 16, 64, 8, 64, 24, [600, 250], 0), (40, 5, 16, 8, 256, 16, [600, 250], 0)], ids=str)
def test_attention_wait_runs_out_and_the_next_call_is_right(c):
    """A limit far below a wait's time: MOE_DEV_TIMEOUT is reported, the copies
    and products in flight are waited for, the next call is right.  The long
    wait: each CTA has several sequences, and a last value that is not finite
    has a sequence's earlier rows summed anew, key by key, meanwhile the next
    sequence's weights are waited for."""
    c = c[:6] + ((c[6] * 20),) + c[7:]
    st, window = attention_case(c, 74)
    d = to_dev(st)
    v = d["v_cache"].clone()
    for s, n in enumerate(c[6]):
        v[st["block_table"][s, (n - 1) // c[5]], :, (n - 1) % c[5]] = float("nan")
    try:
        mm.moe_set_wait_limit_ns(1)
        mm.block_attention(**{**d, "v_cache": v}, window=window)
        assert mm.moe_get_device_status() == (5, 4)
    finally:
        mm.moe_set_wait_limit_ns(0)
        mm.moe_clear_device_status()
    check_attention(st, window, mm.block_attention(**d, window=window))


def test_attention_same_bits_again_and_on_another_stream():
    st, window = attention_case((6, 8, 16, 2, 128, 16, [1500, 20, 900, 0, 8, 400], 0), 71)
    d = to_dev(st)
    first = mm.block_attention(**d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = mm.block_attention(**d, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, second)
    ws = mm.alloc_attention_workspace(6, 8, 16, 2, 128, DEV)
    for fill in (0, 255):
        ws.fill_(fill)
        assert torch.equal(first, mm.block_attention(**d, workspace=ws))
    check_attention(st, window, first)


# ----------------------------------------------------------------- sampling --

def check_sample(logits, u=None, **f):
    dev = {k: v.to(DEV) for k, v in f.items()}
    token, probs = mm.block_sample(logits.to(DEV), None if u is None else u.to(DEV), **dev, with_probs=True)
    want_t, want_p = osam.block_sample(logits.double().numpy(), None if u is None else u.numpy(),
                                       **{k: v.numpy() for k, v in f.items()})
    p = f64(probs)
    assert np.array_equal(p > 0, want_p > 2.0 ** -150) or \
        np.array_equal((p > 0)[abs(want_p - 2.0 ** -149) > 2.0 ** -149], (want_p > 0)[abs(want_p - 2.0 ** -149) > 2.0 ** -149])
    assert (abs(p - want_p) <= 2.0 ** -22 * want_p + 2.0 ** -149).all()
    if u is not None:
        assert np.array_equal(token.cpu().numpy(), want_t)
        only, none = mm.block_sample(logits.to(DEV), u.to(DEV), **dev)
        assert none is None and torch.equal(only, token)
    return token, probs


def uniforms(shape, seed):
    return torch.randint(0, 1 << 24, shape, generator=torch.Generator().manual_seed(seed)).float() * 2.0 ** -24


FILTERS = {
    "none": {}, "temperature": dict(temperature=[0.5, 1.0, 2.0, 0.0, -1.0, float("nan")]),
    "top_k": dict(top_k=[1, 2, 17, 0, -3, 100000]),
    "top_p": dict(top_p=[0.9, 0.5, 0.0, 1.0, 0.99999, float("nan")]),
    "min_p": dict(min_p=[0.1, 0.5, 1.0, 2.0, 0.0, float("nan")]),
    "all": dict(temperature=[0.7, 1.3, 0.9, 0.0, 1.0, 1e-6], top_k=[50, 3, 0, 5, 1000, 7],
                top_p=[0.9, 0.95, 0.5, 0.3, 1.0, 0.8], min_p=[0.01, 0.0, 0.02, 0.5, 0.001, 0.1]),
}


def filters(name):
    return {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32)
            for k, v in FILTERS[name].items()}


@pytest.mark.parametrize("name", list(FILTERS))
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4099])
def test_sample(name, V):
    g = torch.Generator().manual_seed(V)
    logits = torch.randn((6, 3, V), generator=g) * 2
    check_sample(logits, uniforms((6, 3), V + 1), **filters(name))


@pytest.mark.parametrize("name", list(FILTERS))
def test_sample_ties(name):
    """bf16-valued logits, few distinct values, all equal: what is kept of
    equal logits goes by index."""
    g = torch.Generator().manual_seed(7)
    z = torch.randn((6, 4, 2500), generator=g) * 2
    z[:, 0] = z[:, 0].to(torch.bfloat16).float()
    z[:, 1] = z[:, 1].round()
    z[:, 2] = 1.25
    z[:, 3] = -z[:, 3].abs().round() * 0.0 - (z[:, 3] > 1).float()      # +0, -0 and -1
    check_sample(z, uniforms((6, 4), 8), **filters(name))


@pytest.mark.parametrize("name", list(FILTERS))
def test_sample_masked_and_infinite(name):
    """-infinity and NaN have no mass, +infinity all of it, the type's lowest
    value is an ordinary (weightless) logit."""
    g = torch.Generator().manual_seed(9)
    z = torch.randn((6, 5, 300), generator=g) * 2
    z[:, 0][torch.rand((6, 300), generator=g) < 0.95] = -math.inf
    z[:, 0, 11] = 0.5
    z[:, 1, ::3] = float("nan")
    z[:, 2, 17], z[:, 2, 200] = math.inf, math.inf
    z[:, 3] = torch.finfo(torch.float32).min
    z[:, 4, 50:] = torch.finfo(torch.float32).min
    check_sample(z, uniforms((6, 5), 10), **filters(name))
    assert mm.moe_get_device_status() == (0, 0)


def test_sample_rows_without_mass():
    z = torch.randn((2, 2, 64))
    z[0, 1] = -math.inf
    z[1, 0] = float("nan")
    check_sample(z, uniforms((2, 2), 1), top_k=i32([5, 0]), top_p=torch.tensor([0.5, 0.5]))
    assert mm.moe_get_device_status() == NO_MASS


@pytest.mark.parametrize("k", [127, 128, 129, 2000, 2048, 2049, 6000])
def test_sample_top_k_sizes(k):
    """Around the sizes where the selection changes its way, without ties, with
    some and with thousands at the border."""
    V = 20011
    z = torch.randn((1, 3, V), generator=torch.Generator().manual_seed(k)) * 2
    z[:, 1] = z[:, 1].to(torch.bfloat16).float()
    z[:, 2] = z[:, 2].round()
    for f in (dict(top_k=i32([k])), dict(top_k=i32([k]), top_p=torch.tensor([0.7])),
              dict(top_k=i32([k]), top_p=torch.tensor([0.9]), min_p=torch.tensor([0.02]))):
        check_sample(z, uniforms((1, 3), k), **f)


def test_sample_largest_vocabulary_and_heavy_ties():
    V = 393216
    z = torch.randn((1, 3, V), generator=torch.Generator().manual_seed(12)) * 2
    z[:, 1] = z[:, 1].round()
    z[:, 2] = 0.0
    for f in ({}, dict(top_p=torch.tensor([0.9])), dict(min_p=torch.tensor([0.3])),
              dict(top_k=i32([100000]), top_p=torch.tensor([0.6]))):
        check_sample(z, uniforms((1, 3), 13), **f)


def test_sample_many_rows():
    """More rows than one launch's grid takes."""
    S, K, V = 23000, 3, 9
    z = torch.randn((S, K, V), generator=torch.Generator().manual_seed(14))
    u = uniforms((S, K), 15)
    token, probs = mm.block_sample(z.to(DEV), u.to(DEV), with_probs=True)
    z64 = z.double().numpy()
    w = np.exp(z64 - z64.max(-1, keepdims=True))
    W = np.floor(w * 2.0 ** 40)
    m = np.floor(W.sum(-1) * u.double().numpy())
    want = (np.cumsum(W, -1) > m[..., None]).argmax(-1)
    p = w / w.sum(-1, keepdims=True)
    assert (abs(f64(probs) - p) <= 2.0 ** -22 * p).all()
    # (numpy's exponential may differ in the last unit of 2^40: a draw on the border)
    border = (abs(np.cumsum(W, -1) - m[..., None]) <= V).any(-1)
    assert np.array_equal(token.cpu().numpy()[~border], want[~border]) and border.mean() < 1e-6


def test_sample_extreme_temperatures():
    z = torch.randn((6, 2, 3001), generator=torch.Generator().manual_seed(16)) * 2
    t = torch.tensor([1e-30, 1e30, 1e-42, math.inf, 3.4e38, 1e-3])
    check_sample(z, uniforms((6, 2), 17), temperature=t)
    check_sample(z, uniforms((6, 2), 18), temperature=t, top_p=torch.full((6,), 0.8), top_k=i32([9] * 6))
    z[:, :, ::5] = torch.finfo(torch.float32).min          # masked: no weight at any temperature
    check_sample(z, uniforms((6, 2), 19), temperature=t)


def test_sample_uniforms_outside_their_range():
    """They count as the nearest one inside: a token is always drawn."""
    z = torch.randn((4, 1, 500), generator=torch.Generator().manual_seed(20)) * 2
    u = torch.tensor([[1.0], [7.5], [-0.25], [float("nan")]])
    token, _ = mm.block_sample(z.to(DEV), u.to(DEV), top_k=i32([0, 30, 30, 0]).to(DEV))
    inside = torch.tensor([[1 - 2.0 ** -24], [1 - 2.0 ** -24], [0.0], [1 - 2.0 ** -24]])
    want, _ = osam.block_sample(z.double().numpy(), inside.numpy(), top_k=np.array([0, 30, 30, 0]))
    assert np.array_equal(token.cpu().numpy(), want)


def test_sample_exact_borders():
    """Equal masses put the draw's borders at u = v / V exactly, and top-p's at
    p = n / V."""
    V = 1 << 12
    u = torch.tensor([[0.0, 0.25, 0.25 - 2.0 ** -24, 0.5, 1 - 2.0 ** -24]])
    z = torch.zeros((1, 5, V))
    t, _ = check_sample(z, u)
    assert t.tolist() == [[0, V // 4, V // 4 - 1, V // 2, V - 1]]
    t, _ = check_sample(z, u, top_p=torch.tensor([0.5]))
    assert t[0, 4] == V // 2 - 1
    t, _ = check_sample(z, u, top_p=torch.tensor([0.5]), top_k=i32([V // 4]))
    assert t[0, 4] == V // 8 - 1


@pytest.mark.parametrize("V", [32000, 50257, 152064, 300001])
def test_sample_vocabularies(V):
    """Vocabulary sizes of the verify workloads and odd ones, every filter."""
    g = torch.Generator().manual_seed(V)
    z = torch.randn((6, 1, V), generator=g) * 2
    z[::2] = z[::2].to(torch.bfloat16).float()
    check_sample(z, uniforms((6, 1), 3), **filters("all"))
    check_sample(z, uniforms((6, 1), 4), **filters("top_p"))


def test_sample_flat_and_steep():
    """Rows at the filters' extremes: all mass on one token, a flat row, a row
    whose logits differ by single float steps, one of large magnitude."""
    V = 3001
    z = torch.zeros((6, 4, V))
    z[:, 0, 77] = 200.0
    z[:, 1] = torch.linspace(-1e-3, 1e-3, V)
    z[:, 2] = 1.0 + torch.arange(V) * 2.0 ** -23
    z[:, 3] = 1e30 * torch.randn(V, generator=torch.Generator().manual_seed(2))
    for name in FILTERS:
        check_sample(z, uniforms((6, 4), 5), **filters(name))


def test_sampled_tokens_follow_the_probabilities():
    """10^5 draws of one filtered row against its probabilities: chi-square over
    the kept tokens below the 0.001 quantile (37.7 at 15 degrees of freedom)."""
    n, V = 100_000, 64
    row = torch.randn(V, generator=torch.Generator().manual_seed(4)) * 1.5
    z = row.expand(n, 1, V).contiguous()
    token, probs = mm.block_sample(z.to(DEV), uniforms((n, 1), 6).to(DEV), with_probs=True,
                                   top_k=torch.full((n,), 16, dtype=torch.int32, device=DEV))
    p = f64(probs[0, 0])
    count = np.bincount(token.cpu().numpy().ravel(), minlength=V)
    assert (count[p == 0] == 0).all() and (p > 0).sum() == 16
    assert ((count - n * p) ** 2 / np.where(p > 0, n * p, 1)).sum() < 37.7


# ------------------------------------------------------ together, and graphs --

def verify_step(st, out):
    """Append, attention, draft and target distributions, acceptance."""
    q = mm.block_kv_append(st["qkv"], st["kv_len"], st["table"], st["k"], st["v"], st["cs"],
                           st["qw"], st["kw"], q_out=out["q"])
    mm.block_attention(q, st["k"], st["v"], st["table"], st["kv_len"], out=out["o"], workspace=out["ws"])
    K = st["draft_logits"].shape[1]
    mm.block_sample(st["draft_logits"], st["u_draft"], temperature=st["t"], token=out["draft"],
                    probs=out["qp"])
    mm.block_sample(st["target_logits"], temperature=st["t"], top_k=st["top_k"], top_p=st["top_p"],
                    probs=out["pp"])
    mm.block_accept_rejection_bonus(out["pp"], out["qp"], out["draft"], st["u_acc"], st["u_res"],
                                    out["acc"], out["next"])
    return K


def step_state(seed, S=6, K=8, Hq=16, Hkv=2, D=128, page=16, V=2000):
    N = K + 1
    lens = [9, 0, 40, 333, 128, 700][:S]
    pages = sum(-(-n // page) for n in lens) + 2
    z = torch.randn((S, N, V), generator=torch.Generator().manual_seed(seed)) * 2
    st = dict(qkv=bf16((S, N, Hq + 2 * Hkv, D), seed), kv_len=i32(lens),
              table=torch.clamp(i32(tables(lens, page, pages, seed)), min=0),
              k=bf16((pages, Hkv, page, D), seed + 1), v=bf16((pages, Hkv, page, D), seed + 2),
              cs=cos_sin(800, D), qw=bf16((D,), seed + 3), kw=bf16((D,), seed + 4),
              target_logits=z, draft_logits=(z[:, :K] + 0.3 * torch.randn((S, K, V))).contiguous(),
              t=torch.tensor([0.7, 1.0, 0.0, 1.2, 0.9, 1.0][:S]), top_k=i32([0, 50, 0, 200, 0, 0][:S]),
              top_p=torch.tensor([1.0, 0.9, 1.0, 0.95, 0.9, 1.0][:S]),
              u_draft=uniforms((S, K), seed + 5), u_acc=uniforms((S, K), seed + 6),
              u_res=uniforms((S,), seed + 7))
    st = to_dev(st)
    e = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device=DEV)
    out = dict(q=e(S, N, Hq, D), o=e(S, N, Hq, D), ws=mm.alloc_attention_workspace(S, N, Hq, Hkv, D, DEV),
               draft=e(S, K, dt=torch.int32), qp=e(S, K, V, dt=torch.float32),
               pp=e(S, N, V, dt=torch.float32), acc=e(S, dt=torch.int32), next=e(S, dt=torch.int32))
    return st, out


def check_step(st, before, out):
    h = {k: v.cpu() for k, v in st.items()}
    q, k, v = np.zeros(out["q"].shape), f64(before["k"]), f64(before["v"])
    oatt.kv_append(f64(h["qkv"]), h["kv_len"].numpy(), h["table"].numpy(), k, v, q, f64(h["cs"]),
                   f64(h["qw"]), f64(h["kw"]))
    # each stage against the oracle on the stage's own inputs
    assert (abs(f64(out["q"]) - q) <= HALF * abs(q) + 2.0 ** -15 * abs(q).max()).all()
    check_attention(dict(q=out["q"].cpu(), k_cache=h["k"], v_cache=h["v"], block_table=h["table"],
                         kv_len=h["kv_len"]), 0, out["o"])
    f = {n: h[n].numpy() for n in ("top_k", "top_p")}
    draft, qp = osam.block_sample(h["draft_logits"].double().numpy(), h["u_draft"].numpy(),
                                  temperature=h["t"].numpy())
    _, pp = osam.block_sample(h["target_logits"].double().numpy(), temperature=h["t"].numpy(), **f)
    assert np.array_equal(out["draft"].cpu().numpy(), draft)
    for got, want in ((out["qp"], qp), (out["pp"], pp)):
        assert (abs(f64(got) - want) <= 2.0 ** -22 * want + 2.0 ** -149).all()
    acc, nxt = oacc.rejection_bonus(out["pp"].cpu().numpy(), out["qp"].cpu().numpy(), draft,
                                    h["u_acc"].numpy(), h["u_res"].numpy())
    assert np.array_equal(out["acc"].cpu().numpy(), acc) and np.array_equal(out["next"].cpu().numpy(), nxt)
    assert (acc > 0).any()
    assert mm.moe_get_device_status() == (0, 0)


def test_verify_step_together():
    st, out = step_state(101)
    before = {k: st[k].clone() for k in ("k", "v")}
    verify_step(st, out)
    check_step(st, before, out)


def test_verify_step_captured_and_replayed():
    """One graph, replayed on new inputs and lengths copied into its tensors;
    two graphs that share the attention workspace, replayed in turn."""
    st, out = step_state(201)
    st2, out2 = step_state(301)
    out2["ws"] = out["ws"]
    verify_step(st, out)
    verify_step(st2, out2)
    torch.cuda.synchronize()
    graphs = []
    for s, o in ((st, out), (st2, out2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            verify_step(s, o)
        graphs.append(g)
    fresh, _ = step_state(401)
    fresh["kv_len"] = fresh["kv_len"].flip(0).contiguous()
    fresh["table"] = fresh["table"].flip(0).contiguous()
    for k in st:
        st[k].copy_(fresh[k])
    for o in (out, out2):
        for k, t in o.items():
            if k != "ws":
                t.zero_()
    b1 = {k: st[k].clone() for k in ("k", "v")}
    b2 = {k: st2[k].clone() for k in ("k", "v")}
    for _ in range(2):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    check_step(st, b1, out)
    check_step(st2, b2, out2)
    del graphs


# ---------------------------------------------------------- binding's checks --

def test_binding_refuses():
    st, _ = attention_case(ATTENTION[2], 1)
    d = to_dev(st)
    call = lambda **kw: mm.block_attention(**{**d, **kw})
    with pytest.raises(ValueError, match="v_cache"):
        call(v_cache=d["v_cache"][:-1])
    with pytest.raises(ValueError, match="contiguous"):
        call(q=d["q"].transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError, match="kv_len"):
        call(kv_len=d["kv_len"].long())
    with pytest.raises(ValueError, match="kv_len"):
        call(kv_len=d["kv_len"][:2])
    with pytest.raises(ValueError, match="k_cache"):
        call(k_cache=d["k_cache"][..., :64].contiguous(), v_cache=d["v_cache"][..., :64].contiguous())
    with pytest.raises(ValueError, match="CUDA"):
        call(block_table=st["block_table"])
    with pytest.raises(mm.MoeError) as e:
        call(window=-1)
    assert e.value.status == 1
    with pytest.raises(mm.MoeError) as e:
        call(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 4
    z = torch.zeros((2, 3, 8), device=DEV)
    with pytest.raises(ValueError, match="u must be"):
        mm.block_sample(z, torch.zeros((3, 2), device=DEV))
    with pytest.raises(ValueError, match="top_k"):
        mm.block_sample(z, top_k=torch.zeros(2, device=DEV), with_probs=True)
    with pytest.raises(mm.MoeError):
        mm.block_sample(z)
