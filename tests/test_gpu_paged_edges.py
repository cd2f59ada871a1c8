"""GPU tests of the paged cache at the corners of its contract: gates of both
signs, infinite values and sinks, sums past fp32, a stack with entries that are
no pages, the largest batch, and the forms that the ordinary cases pass by."""
import math

import numpy as np
import pytest
import torch

from channel_decay_softmax_b200 import _lib as L
from channel_decay_softmax_b200 import api
from oracle import wall_oracle as wo
from tests import paged_reference as ref
from tests import test_gpu_paged as tp
from tests.helpers import assert_fwd, max_abs

pytestmark = pytest.mark.gpu

DEV, BF, F32 = tp.DEV, tp.BF, tp.F32
_i32 = tp._i32


def _status_ok():
    assert L.wall_get_status() == L.WALL_OK


# Kernels that the attention of 40 rows, of up to eight and of one may take.
ROUTES = [(4, 2, 128, BF), (2, 1, 64, BF), (1, 1, 128, BF), (8, 1, 64, BF), (12, 1, 64, BF),
          (2, 1, 64, F32)]


def _cache_of(P, q, k, new, H, V, PS, dt, seed=0):
    """One request's cache and its last `new` query rows, from its prefix P
    [n, HQ, K] (powers of two), queries q [new, HQ, K] and keys k [n, HQ, K]."""
    n, HQ, K = P.shape
    gen = torch.Generator().manual_seed(700 + seed)
    cu, kv, table, _, NP = tp._batch([new], [n - new], PS, seed)
    kp, r = torch.zeros(NP, HQ, PS, K), torch.zeros(NP, HQ, K, dtype=torch.int32)
    p = torch.empty(n, HQ, K)
    for j in range(n):
        page = int(table[0, j // PS])
        if j % PS == 0:
            r[page] = torch.floor(P[j] + 0.5).int()
        p[j] = P[j] - r[page]
        kp[page, :, j % PS] = k[j] * torch.exp2(-p[j])
    assert p.abs().max() <= 100  # what a page may hold
    return dict(q=q.to(dt).to(DEV), p=p[n - new:].contiguous().to(DEV), k_pages=kp.to(dt).to(DEV),
                v_pages=tp._rand(gen, NP, H, PS, V, dtype=dt), r_pages=r.to(DEV)), cu, kv, table


def _attn(x, cu, kv, table, **kw):
    return api.wall_paged_attn(x["q"], x["p"], _i32(cu), _i32(kv), _i32(table), x["k_pages"],
                               x["v_pages"], x["r_pages"], return_lse=True, **kw)


# --------------------------------------------------------------- the largest batches

def test_attn_flags_of_the_largest_batches():
    """More (block, head) places than 31 bits count: a NaN value of the last
    request marks that request's unit, and its other rows stay."""
    N, HQ, H, K, PS, n = (1 << 19) + 4, 4096, 512, 64, 32, 9
    gen = torch.Generator(device=DEV).manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(BF)
    x = dict(q=rand(n, HQ, K), p=torch.zeros(n, HQ, K, device=DEV), k_pages=rand(1, HQ, PS, K),
             v_pages=rand(1, H, PS, K), r_pages=torch.zeros(1, HQ, K, dtype=torch.int32, device=DEV))
    x["v_pages"][:, :, n - 1] = math.nan
    args = lambda N: (x["q"], x["p"],
                      torch.cat([torch.zeros(N, dtype=torch.int32, device=DEV), _i32([n])]),
                      torch.cat([torch.zeros(N - 1, dtype=torch.int32, device=DEV), _i32([n])]),
                      torch.zeros(N, 1, dtype=torch.int32, device=DEV), x["k_pages"], x["v_pages"],
                      x["r_pages"])
    want = api.wall_paged_attn(*args(1))
    got = api.wall_paged_attn(*args(N))
    _status_ok()
    assert torch.isfinite(want[:n - 1]).all() and torch.isnan(want[n - 1]).all()
    assert torch.equal(got[:n - 1], want[:n - 1]) and torch.isnan(got[n - 1]).all()
    del got
    torch.cuda.empty_cache()
