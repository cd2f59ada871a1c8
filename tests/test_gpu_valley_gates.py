"""Training with gates of both signs whose channels fall inside one 128-row
block, lie lower still at the next block's anchor and rise again inside that
block: tokens at both ends see one another although the blocks' anchors are
130 powers of two apart, below what one bf16 factor holds."""
import numpy as np
import pytest
import torch

from channel_decay_softmax_b200 import _lib as L
from channel_decay_softmax_b200 import api
from oracle import wall_oracle as wo
from tests.helpers import assert_fwd, assert_grad

pytestmark = pytest.mark.gpu

DEV, BF = "cuda", torch.bfloat16
NAMES = ("dq", "dk", "dv", "dg")


def _valley(T, at=128, fall=68.0, rise=68.0):
    """Prefix: down by `fall` in the block before row `at`, 130 lower than its
    start there, up by `rise` over the next 100 rows."""
    return np.interp(np.arange(T), [at - 128, at - 10, at - 1, at, at + 100],
                     [0.0, -fall, -fall, -130.0, -130.0 + rise])


def _inputs(K, lens, seed=1, HQ=4, H=2):
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens)
    r = lambda *s: torch.randn(1, *s, generator=gen)
    x = dict(q=r(T, HQ, K), k=r(T, H, K), v=r(T, H, K), dO=r(T, HQ, K),
             g=-0.01 * r(T, HQ, K).abs())
    at = 0
    for n in lens:
        if n > 200:
            step = np.diff(np.concatenate([[0.0], _valley(n)])) * np.log(2)
            g = torch.tensor(step).float()[:, None, None]
            x["g"][0, at:at + n, HQ // 2:, ::8] = g      # kv heads from the middle on
            x["q"][0, at:at + n, HQ // 2:, ::8] /= 16
            x["k"][0, at + 128:at + n, H // 2:, ::8] = 0  # the valley's floor: 2^68 below the rows
        at += n
    return {n: t.to(BF) for n, t in x.items()}


def _check(x, o, lse, grads, ref, what):
    assert_fwd(BF, o, ref["o"], lse, ref["lse"], what=what)
    for name, got in zip(NAMES, grads):
        assert_grad(BF, name, got, ref[name], what=what)
    assert L.wall_get_status() == L.WALL_OK


@pytest.mark.parametrize("K", [64, 128])
@pytest.mark.parametrize("lens,window", [([229], 0), ([300, 100, 260], 0), ([229], 150)])
def test_valley(K, lens, window):
    xc = _inputs(K, lens)
    cu = np.concatenate([[0], np.cumsum(lens)]) if len(lens) > 1 else None
    kw = dict(scale=K ** -0.5, window_size=window or None)
    ref = wo.backward(xc["q"], xc["k"], xc["v"], xc["g"], xc["dO"], cu_seqlens=cu, **kw)
    x = {n: t.to(DEV) for n, t in xc.items()}
    if cu is not None:
        kw["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    P = api.prefix_cumsum(x["g"], cu_seqlens=kw.get("cu_seqlens"))
    a = (x["q"], x["k"], x["v"])
    o, lse = api.wall_attn_fwd(*a, P, **kw)
    for store_ds in (True, False):
        grads = api.wall_attn_bwd(x["dO"], *a, P, o, lse, store_ds=store_ds, **kw)
        _check(x, o, lse, grads, ref, f"from P, store_ds={store_ds}")
    o, lse, P, ws = api.wall_attn_fwd_gate(*a, x["g"], return_workspace=True, **kw)
    grads = api.wall_attn_bwd(x["dO"], *a, P, o, lse, fwd_workspace=ws, **kw)
    _check(x, o, lse, grads, ref, "gate call")


def test_rise_and_fall_in_blocks_far_apart():
    """The fall and the rise of a unit in blocks that other CTAs form, in both
    orders of time, and rises or falls alone, which stay on the tensor cores."""
    K, T = 64, 900
    for fall, rise in ((68.0, 68.0), (90.0, 40.0), (40.0, 90.0), (0.0, 60.0), (95.0, 0.0)):
        gen = torch.Generator().manual_seed(5)
        r = lambda *s: torch.randn(1, *s, generator=gen)
        xc = dict(q=r(T, 4, K), k=r(T, 2, K), v=r(T, 2, K), dO=r(T, 4, K), g=-0.01 * r(T, 4, K).abs())
        P = np.interp(np.arange(T), [0, 118, 127, 640, 740, T], [0.0, -fall, -fall, -130.0, -130.0 + rise,
                                                                   -130.0 + rise])
        xc["g"][0, :, 2, ::8] = torch.tensor(np.diff(np.concatenate([[0.0], P])) * np.log(2)).float()[:, None]
        xc["q"][0, :, 2, ::8] /= 16
        xc["k"][0, 128:, 1, ::8] = 0
        xc = {n: t.to(BF) for n, t in xc.items()}
        ref = wo.backward(xc["q"], xc["k"], xc["v"], xc["g"], xc["dO"], scale=K ** -0.5)
        x = {n: t.to(DEV) for n, t in xc.items()}
        o, lse, Pd, ws = api.wall_attn_fwd_gate(x["q"], x["k"], x["v"], x["g"], K ** -0.5,
                                                return_workspace=True)
        grads = api.wall_attn_bwd(x["dO"], x["q"], x["k"], x["v"], Pd, o, lse, K ** -0.5,
                                  fwd_workspace=ws)
        _check(x, o, lse, grads, ref, f"fall {fall} rise {rise}")
