"""GPU checks of the block's append, attention and sampling where several of
their parts meet: rows that fill a block in part over many tiles, values that
are not finite, masses at a filter's border.

The attention is compared with `attention64`, the definition in float64 on the
device (the oracle's loops are too slow for these sizes), under the tolerance
that test_gpu_block.py derives.
"""
import threading

import numpy as np
import pytest
import torch

import mxfp4_moe_block_b200 as mm
from test_gpu_block import (DEV, EPS, HALF, attention_case, check_step, clean_status, cos_sin,  # noqa: F401
                            step_state, to_dev, verify_step)

pytestmark = pytest.mark.gpu


def attention64(d, window, scale=None):
    """(out, spread) in float64: softmax of the keys a token sees, and the weighted
    mean of |v|, which rounding errors of the weights scale with."""
    S, N, Hq, D = d["q"].shape
    pages, Hkv, page, _ = d["k_cache"].shape
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros((S, N, Hq, D), dtype=torch.float64, device=DEV)
    spread = torch.zeros_like(out)
    for s, n in enumerate(d["kv_len"].tolist()):
        lo = max(0, n - N - window + 1) if window else 0
        j = torch.arange(lo, max(n, 0), device=DEV)
        if len(j) == 0:
            continue
        at = d["block_table"][s].long()[j // page]
        k, v = (d[c][at, :, j % page].double().transpose(0, 1) for c in ("k_cache", "v_cache"))   # [Hkv, n, D]
        q = d["q"][s].double().view(N, Hkv, Hq // Hkv, D)
        pos = (n - N + torch.arange(N, device=DEV))[:, None]
        see = (j <= pos) & (j > pos - window if window else j >= 0)                             # [N, n]
        z = torch.einsum("ihgd,hnd->hgin", q, k) * scale
        z = z.masked_fill(~see, -torch.inf)
        e = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-1e300))
        p = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
        for to, x in ((out, v), (spread, v.abs())):
            to[s] = torch.einsum("hgin,hnd->ihgd", p, x).reshape(N, Hq, D)
    return out, spread


def limit(d, want, spread, scale=None):
    """The tolerance of the attention's outputs (see test_gpu_block.py)."""
    D = d["q"].shape[-1]
    big = d["q"].double().norm(dim=-1).max() * torch.nan_to_num(d["k_cache"].float()).norm(dim=-1).max()
    dz = (D + 4) * EPS * (D ** -0.5 if scale is None else scale) * big
    return HALF * want.abs() + (HALF + 4 * dz + 2.0 ** -17) * spread


def check64(d, window, got):
    want, spread = attention64(d, window)
    over = (got.double() - want).abs() - limit(d, want, spread)
    assert (over <= 0).all(), float(over.max())
    assert mm.moe_get_device_status() == (0, 0)


# ------------------------------------------------ rows that fill a block in part --

@pytest.mark.parametrize("c", [
    # N, Hq, Hkv, D, page, window: rows to a key/value head, of them in the last block
    (33, 10, 2, 64, 16, 0),        # 165, 37
    (16, 5, 1, 64, 5, 0),          # 80
    (24, 7, 1, 64, 64, 1000),      # 168, 40
    (17, 8, 1, 128, 32, 0),        # 136, 8
    (16, 10, 2, 128, 24, 700),     # 80
    (20, 8, 1, 128, 7, 0),         # 160, 32
    (33, 14, 2, 128, 128, 0),      # 231, 103 (every warp has rows)
    (17, 16, 2, 256, 16, 0),       # 136, 8
    (33, 6, 1, 256, 64, 500),      # 198, 70
], ids=str)
def test_attention_rows_that_fill_a_block_in_part(c):
    """Softmax warps without rows beside those that have some, over segments of many
    tiles: each tile's weights are complete before its product with the values."""
    N, Hq, Hkv, D, page, window = c
    lens = [600 + (s * 1709) % 3400 for s in range(64)]
    st, _ = attention_case((64, N, Hq, Hkv, D, page, lens, window), 91)
    d = to_dev(st)
    ws = mm.alloc_attention_workspace(64, N, Hq, Hkv, D, DEV)
    outs = [mm.block_attention(**d, window=window, workspace=ws) for _ in range(6)]
    d = {k: torch.nan_to_num(v) if v.is_floating_point() else v for k, v in d.items()}
    check64(d, window, outs[0])
    assert all(torch.equal(outs[0], o) for o in outs[1:])


# --------------------------------------------------- values that are not finite --

@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("N,Hq,Hkv,D", [
    (1, 8, 1, 128), (8, 8, 2, 64), (12, 8, 2, 64), (16, 16, 2, 128), (33, 4, 1, 64),
    (5, 6, 2, 256), (10, 8, 2, 256), (4, 32, 2, 128)], ids=str)
def test_attention_infinite_values_come_out_as_such(N, Hq, Hkv, D, window):
    """An infinite value is the result of every token that sees it, whatever the
    number of rows; with one of each sign the result is NaN; a token that does not
    see it is not touched."""
    lens, page = [700, 90, 2000], 16
    st, _ = attention_case((3, N, Hq, Hkv, D, page, lens, window), 92)
    d = {k: torch.nan_to_num(v) if v.is_floating_point() else v for k, v in to_dev(st).items()}
    inf = float("inf")
    # (key, dims, value): two that all tokens see, one that the last alone sees
    marks = lambda n: [(n - N - 3, 5, inf), (n - N - 40, 6, -inf), (n - N - 3, 4, inf), (n - N - 40, 4, -inf),
                       (n - 1, 3, inf)]
    clean = d["v_cache"].clone()
    for s, n in enumerate(lens):
        for key, dim, value in marks(n):
            d["v_cache"][d["block_table"][s, key // page], :, key % page, dim::7] = value
            clean[d["block_table"][s, key // page], :, key % page, dim::7] = 0
    want, spread = attention64({**d, "v_cache": clean}, window)
    lim = limit(d, want, spread)
    for s in range(3):
        want[s, :, :, 5::7], want[s, :, :, 6::7], want[s, :, :, 4::7] = inf, -inf, float("nan")
        want[s, N - 1, :, 3::7] = inf
    got = mm.block_attention(**d, window=window).double()
    assert mm.moe_get_device_status() == (0, 0)
    fine = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()])
    assert ((got - want).abs()[fine] <= lim[fine]).all()


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(3, 8, 2, 128), (12, 8, 2, 64), (16, 16, 2, 128), (33, 4, 1, 64), (5, 6, 2, 256)])
def test_attention_keys_that_are_not_finite_reach_no_other_token(N, Hq, Hkv, D, value):
    """The last token's key: a score of +infinity or NaN makes the last token's result
    NaN, one of -infinity weighs nothing; the other tokens are as without it."""
    lens, page = [700, 90, 2000], 16
    st, _ = attention_case((3, N, Hq, Hkv, D, page, lens, 0), 94)
    d = {k: torch.nan_to_num(v) if v.is_floating_point() else v for k, v in to_dev(st).items()}
    lim = limit(d, *attention64(d, 0))
    for s, n in enumerate(lens):
        d["k_cache"][d["block_table"][s, (n - 1) // page], :, (n - 1) % page, 0] = value
    want, _ = attention64(d, 0)
    got = mm.block_attention(**d).double()
    assert mm.moe_get_device_status() == (0, 0)
    assert torch.equal(got.isnan(), want.isnan()) and want[:, -1].isnan().any() and not want[:, :-1].isnan().any()
    assert ((got - want).abs() <= lim)[~want.isnan()].all()


@pytest.mark.parametrize("N,Hq,D", [(16, 64, 128), (16, 64, 64), (8, 64, 256)], ids=str)
def test_attention_summing_anew_outlasts_the_wait_limit(N, Hq, D):
    """A value that is not finite in a long cache: its sequence's other rows are summed
    anew key by key, while the waits for the next sequence's tiles run on.  They are not
    cut short by a limit that the summing as a whole passes.  (Of one sequence and head
    it takes 36 to 92 ms, and up to 10 ms to a beat, 32768 keys of a warp.)"""
    S, Hkv, page, n = 40, 8, 64, 16384
    st, _ = attention_case((1, N, Hq, Hkv, D, page, [n], 0), 93)
    d = {k: torch.nan_to_num(v) if v.is_floating_point() else v for k, v in to_dev(st).items()}
    d["q"], d["block_table"], d["kv_len"] = (t.repeat_interleave(S, 0) for t in (d["q"], d["block_table"], d["kv_len"]))
    one = {**d, "q": d["q"][:1], "block_table": d["block_table"][:1], "kv_len": d["kv_len"][:1]}
    want, spread = attention64(one, 0)
    lim = limit(d, want, spread)
    d["v_cache"][d["block_table"][0, (n - 1) // page], :, (n - 1) % page] = float("nan")
    try:
        mm.moe_set_wait_limit_ns(15_000_000)
        out = mm.block_attention(**d).double()
        assert mm.moe_get_device_status() == (0, 0)
    finally:
        mm.moe_set_wait_limit_ns(0)
    assert out[:, -1].isnan().all()
    assert ((out[:, :-1] - want[:, :-1]).abs() <= lim[:, :-1]).all()


# -------------------------------------------------- dims that are not rotated --

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 48), (128, 64), (256, 32), (256, 240)])
def test_append_infinities_in_dims_that_are_not_rotated(D, rot, interleaved):
    """Without norms the dims past `rot` pass through, whatever they hold."""
    S, N, Hq, Hkv, page, n = 2, 3, 6, 2, 16, 40
    g = torch.Generator().manual_seed(D + rot)
    qkv = torch.randn((S, N, Hq + 2 * Hkv, D), generator=g).to(torch.bfloat16)
    qkv[..., rot + 1::3] = float("inf")
    qkv[..., rot + 5::9] = -float("inf")
    qkv[..., rot + 6::11] = float("nan")
    cs = cos_sin(n, rot).to(DEV)
    table = torch.arange(S * 3, dtype=torch.int32, device=DEV).view(S, 3)
    kc, vc = (torch.zeros((S * 3, Hkv, page, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = mm.block_kv_append(qkv.to(DEV), torch.full((S,), n, dtype=torch.int32, device=DEV), table, kc, vc,
                           cs, norm=False, interleaved=interleaved).cpu()
    at = torch.arange(n - N, n)
    k = kc.cpu()[table.cpu().long()[:, at // page], :, at % page]                        # [S, N, Hkv, D]
    for got, want in ((q, qkv[:, :, :Hq]), (k, qkv[:, :, Hq:Hq + Hkv])):
        torch.testing.assert_close(got[..., rot:], want[..., rot:], rtol=0, atol=0, equal_nan=True)
    assert q[..., :rot].isfinite().all() and k[..., :rot].isfinite().all()


# ------------------------------------------------------ masses at a filter's border --

def border_logits(temperature, seed):
    """Logits l below a largest one of 0 whose mass W = floor(2^40 exp(l / T)) lies at a
    multiple of 2^16 or one below it, so that a float min_p tells the two apart; those
    with 2^40 exp(l / T) within 0.02 of a whole number are left out (numpy's exponential
    is good to 2^-11 there).  Returns (l, W)."""
    l = -np.random.default_rng(seed).uniform(1e-3, 0.69 * temperature, 1 << 23).astype(np.float32)
    y = np.exp(l.astype(np.float64) / temperature) * 2.0 ** 40
    W = np.floor(y)
    frac, step = y - W, W % 65536
    pick = (frac > 0.02) & (frac < 0.98) & ((step == 0) | (step == 65535))
    return l[pick], W[pick].astype(np.int64)


def kept_second(l, **f):
    """Whether the token of logit l is kept beside one of logit 0."""
    z = torch.zeros((len(l), 1, 5))
    z[:, 0, 3] = torch.from_numpy(l)
    z[:, 0, [0, 2, 4]] = -40.0
    _, probs = mm.block_sample(z.to(DEV), **{k: v.to(DEV) for k, v in f.items()}, with_probs=True)
    return (probs[:, 0, 3] > 0).cpu().numpy()


@pytest.mark.parametrize("T", [1.0, 0.75, 3.0])
@pytest.mark.parametrize("beside", ["alone", "top_k", "top_p"])
def test_sample_masses_at_the_min_p_border(T, beside):
    l, W = border_logits(T, int(T * 4))
    assert len(l) > 100 and (W % 65536 == 0).any() and (W % 65536 != 0).any()
    low = (W + 65535) // 65536                               # min_p 2^24
    f = dict(temperature=torch.full((len(l),), T), min_p=torch.from_numpy(low * 2.0 ** -24).float())
    if beside == "top_k":
        f["top_k"] = torch.full((len(l),), 3, dtype=torch.int32)
    elif beside == "top_p":
        f["top_p"] = torch.full((len(l),), 1 - 2.0 ** -24)
    assert np.array_equal(kept_second(l, **f), W >= low * 65536)


def test_sample_masses_at_the_top_p_border():
    """Two tokens and a float p at which one unit of the second's mass decides whether
    the first alone reaches p of the sum."""
    l = -np.random.default_rng(5).uniform(1e-3, 0.69, 1 << 24).astype(np.float32)
    w = np.exp(l.astype(np.float64))
    p = np.round(2.0 ** 24 / (1 + w)) * 2.0 ** -24
    near = abs(p * (1 + w) - 1) * 2.0 ** 40 < 2
    l, w, p = l[near], w[near], p[near]
    y = w * 2.0 ** 40
    W = np.floor(y)
    stays = lambda m: np.ceil(p * (2.0 ** 40 + m)) > 2.0 ** 40
    pick = (y - W > 0.02) & (y - W < 0.98) & (stays(W - 1) != stays(W + 1))
    assert pick.sum() > 100
    l, p, want = l[pick], p[pick], stays(W)[pick]
    assert want.any() and not want.all()
    for V, f in ((2, {}), (5, dict(top_k=torch.full((len(l),), 2, dtype=torch.int32)))):
        z = torch.full((len(l), 1, V), -60.0)
        z[:, 0, 0], z[:, 0, 1] = 0.0, torch.from_numpy(l)
        f = {k: v.to(DEV) for k, v in dict(f, top_p=torch.from_numpy(p).float()).items()}
        _, probs = mm.block_sample(z.to(DEV), **f, with_probs=True)
        assert np.array_equal((probs[:, 0, 1] > 0).cpu().numpy(), want)


# ------------------------------------------------------------------ host threads --

def test_verify_steps_of_several_host_threads():
    """Four threads, a stream and a workspace each, all three calls."""
    steps = [step_state(500 + i) for i in range(4)]
    before = [{k: st[k].clone() for k in ("k", "v")} for st, _ in steps]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(10):
                    verify_step(*steps[i])
            stream.synchronize()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for (st, out), b in zip(steps, before):
        check_step(st, b, out)
