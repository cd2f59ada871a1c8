"""Decode over caches whose work items have an odd number of 32-key tiles: the
head's two warps then change places from item to item, and neither may take a
stage of the copy ring for a later one's."""
import pytest
import torch

from channel_decay_softmax_b200 import api
from channel_decay_softmax_b200 import _lib as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("HQ,H", [(1, 1), (4, 1), (8, 1)])
@pytest.mark.parametrize("T,C", [(96, 32), (160, 32), (1120, 32), (1056, 64)])
def test_decode_odd_tiles(T, C, HQ, H):
    B, K = 160, 128
    gen = torch.Generator(device="cuda").manual_seed(T + HQ)
    bf = dict(device="cuda", generator=gen, dtype=torch.float32)
    k, v = (torch.randn(B, T, H, K, **bf).bfloat16() for _ in range(2))
    g = (-0.02 * torch.randn(B, T, HQ, K, **bf).abs()).bfloat16()
    q = torch.randn(B, 1, HQ, K, **bf).bfloat16()
    P = api.prefix_cumsum(g)
    kt, rc = api.build_wall_kv_cache(k, P, chunk_size=C)
    call = lambda: api.wall_attn_decode(q, v, P[:, -1:], kt, rc, scale=K ** -0.5, cache_chunk_size=C)
    o, lse = call()
    # the formula in 64 bits, over the cache as it is stored
    R = rc.double().repeat_interleave(C, dim=1)[:, :T]
    s = K ** -0.5 * (q.double() * torch.exp2(P[:, -1:].double() - R) * kt.double()).sum(-1)
    w = torch.softmax(s, dim=1)
    ref = torch.einsum("bth,bthv->bhv", w, v.double().repeat_interleave(HQ // H, dim=2))
    # |o| < 4: half a bf16 step there is 2^-7; the rest is fp32
    assert (o[:, 0].double() - ref).abs().max() <= 2 ** -7 + 1e-4
    for _ in range(20):
        o2, lse2 = call()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert L.wall_get_status() == L.WALL_OK
