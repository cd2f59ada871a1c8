"""Chunks of queries against the decode cache with gates of both signs: keys far
down their cache chunk and rows far up their block, whose anchors are 130
powers of two apart, see one another at up to 2^6."""
import numpy as np
import pytest
import torch

from channel_decay_softmax_b200 import _lib as L
from channel_decay_softmax_b200 import api
from oracle import wall_oracle as wo
from tests.helpers import assert_fwd

pytestmark = pytest.mark.gpu

DEV, BF = "cuda", torch.bfloat16


@pytest.mark.parametrize("K", [64, 128])
@pytest.mark.parametrize("C", [32, 64, 128])
@pytest.mark.parametrize("Tq", [100, 12])
def test_decode_chunk_across_a_valley(K, C, Tq):
    B, HQ, H, T = 2, 4, 2, 228
    gen = torch.Generator().manual_seed(C + Tq)
    r = lambda *s: torch.randn(B, *s, generator=gen)
    q, k, v, g = r(T, HQ, K), r(T, H, K), r(T, H, K), -0.01 * r(T, HQ, K).abs()
    P = np.interp(np.arange(T), [128 - C, 118, 127, 128, T - 1], [0.0, -68.0, -68.0, -130.0, -62.0])
    g[:, :, :, ::8] = torch.tensor(np.diff(np.concatenate([[0.0], P])) * np.log(2)).float()[:, None, None]
    q[..., ::8] /= 16
    k[:, 128:, :, ::8] = 0  # the valley's floor: 2^68 below the rows
    q, k, v, g = (t.to(BF) for t in (q, k, v, g))
    ref, lse_ref = wo.forward(q, k, v, g, scale=K ** -0.5)[:2]
    q, k, v, g = (t.to(DEV) for t in (q, k, v, g))
    P = api.prefix_cumsum(g)
    k_tilde, r_cache = api.build_wall_kv_cache(k, P, chunk_size=C)
    at = T - Tq
    o, lse = api.wall_attn_decode_chunk(q[:, at:], v, P[:, at:].contiguous(), k_tilde, r_cache,
                                        scale=K ** -0.5, cache_chunk_size=C)
    assert L.wall_get_status() == L.WALL_OK
    assert_fwd(BF, o, ref[:, at:], lse, lse_ref[:, at:])
