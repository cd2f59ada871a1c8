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


# ------------------------------------------------------------ gates of both signs

@pytest.mark.parametrize("PS", [32, 64, 128])
@pytest.mark.parametrize("HQ,H,K,dt", ROUTES)
@pytest.mark.parametrize("new", [1, 8, 40])
def test_attn_keys_seen_across_a_valley(new, HQ, H, K, dt, PS):
    """Every eighth channel falls by 68 powers of two over the first page, by 62
    more to the next one and rises by 68 among the rows: keys at the first page's
    end count with up to 2^6, though the pages' anchors are 130 apart."""
    gen = torch.Generator().manual_seed(new + PS)
    n = PS + 40
    t = np.arange(n)
    valley = np.interp(t, [0, PS - 10, PS - 1, PS, n - 1], [0.0, -68.0, -68.0, -130.0, -62.0])
    P = torch.tensor(-0.02 * t).float()[:, None, None].repeat(1, HQ, K)
    P[:, :, ::8] = torch.tensor(valley).float()[:, None, None]
    q, k = torch.randn(new, HQ, K, generator=gen), torch.randn(n, HQ, K, generator=gen)
    q[:, :, ::8] *= 1 / 64 if dt == F32 else 1 / 16
    k[PS:, :, ::8] = 0  # against the valley's floor the rows would see 2^68
    x, cu, kv, table = _cache_of(P, q, k, new, H, K, PS, dt)
    scale = K ** -0.5
    want, lse_want = ref.attn(x["q"], x["p"], cu, kv, torch.tensor(table), x["k_pages"],
                              x["v_pages"], x["r_pages"], PS, scale)
    # the channels matter here: without them the result is another one
    gone = x["q"].clone()
    gone[:, :, ::8] = 0
    other, _ = ref.attn(gone, x["p"], cu, kv, torch.tensor(table), x["k_pages"], x["v_pages"],
                        x["r_pages"], PS, scale)
    assert np.abs(want - other).max() > (1e-3 if dt == F32 else 0.05)
    o, lse = _attn(x, cu, kv, table, scale=scale, max_new=new)
    _status_ok()
    assert_fwd(dt, o, want, lse, lse_want)


def test_attn_long_zigzag():
    """Channels that fall and rise by 60 powers of two every 80 tokens on a slow
    way down, over many pages and several units of rows."""
    HQ, H, K, PS, new, n = 2, 1, 128, 64, 300, 700
    gen = torch.Generator().manual_seed(3)
    t = np.arange(n)
    zig = -0.15 * t + 60.0 * np.abs((t % 80) / 40.0 - 1.0)
    P = torch.tensor(-0.01 * t).float()[:, None, None].repeat(1, HQ, K)
    P[:, :, ::16] = torch.tensor(zig).float()[:, None, None]
    q, k = torch.randn(new, HQ, K, generator=gen), torch.randn(n, HQ, K, generator=gen)
    low = torch.tensor(zig < np.maximum.accumulate(zig[::-1])[::-1] - 4.0)
    k[low, :, ::16] = 0   # keys that a later row would see at more than 2^4
    x, cu, kv, table = _cache_of(P, q, k, new, H, K, PS, BF)
    want, lse_want = ref.attn(x["q"], x["p"], cu, kv, torch.tensor(table), x["k_pages"],
                              x["v_pages"], x["r_pages"], PS, K ** -0.5)
    o, lse = _attn(x, cu, kv, table)
    _status_ok()
    assert_fwd(BF, o, want, lse, lse_want)


# -------------------------------------------------------------- growth past fp32

@pytest.mark.parametrize("PS", [32, 64])
@pytest.mark.parametrize("HQ,H,K,dt", ROUTES)
@pytest.mark.parametrize("new", [1, 8, 40])
def test_attn_growth_past_the_floats(new, HQ, H, K, dt, PS):
    """Channels that gain 80 powers of two a page, up to 2^200 and more between
    a key and a row, where the query or the key is 0: they add nothing."""
    gen = torch.Generator().manual_seed(new + PS)
    n = 2 * PS + 60
    t = torch.arange(n).float()
    P = (-0.02 * t)[:, None, None].repeat(1, HQ, K)
    P[:, :, ::4] = (80.0 / PS * t)[:, None, None]
    q, k = torch.randn(new, HQ, K, generator=gen), torch.randn(n, HQ, K, generator=gen)
    q[:, :, ::8] = 0
    k[:, :, 4::8] = 0
    x, cu, kv, table = _cache_of(P, q, k, new, H, K, PS, dt)
    want, lse_want = ref.attn(x["q"], x["p"], cu, kv, torch.tensor(table), x["k_pages"],
                              x["v_pages"], x["r_pages"], PS, K ** -0.5)
    o, lse = _attn(x, cu, kv, table, max_new=new)
    _status_ok()
    assert_fwd(dt, o, want, lse, lse_want)


# ------------------------------------------------------------------ infinite sinks

@pytest.mark.parametrize("HQ,H,K,dt", ROUTES)
@pytest.mark.parametrize("new,ctx,mx", [([1, 1, 1], [70, 0, 6000], 1), ([3, 8, 1], [70, 5, 6000], 8),
                                        ([40, 20, 1, 150], [70, 0, 3, 900], None)])
def test_attn_sink_of_minus_infinity_is_no_sink(HQ, H, K, dt, new, ctx, mx):
    """A head whose sink is switched off: bit for bit the call without a sink,
    the rows of refused requests (which see nothing) included."""
    x, cu, kv, table = tp._attn_inputs(HQ, H, K, K, 64, dt, new, ctx, refused=(1,), decay=0.002)
    o, lse = _attn(x, cu, kv, table, max_new=mx)
    off = torch.full((HQ,), -math.inf, device=DEV)
    o2, lse2 = _attn(x, cu, kv, table, max_new=mx, sink_bias=off)
    _status_ok()
    assert (o2[cu[1]:cu[2]] == 0).all() and (lse2[cu[1]:cu[2]] == -math.inf).all()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if HQ > 1:  # one head with, the others without
        off[0] = 0.3
        one = torch.full((HQ,), 0.3, device=DEV)
        o3, lse3 = _attn(x, cu, kv, table, max_new=mx, sink_bias=off)
        o4, lse4 = _attn(x, cu, kv, table, max_new=mx, sink_bias=one)
        assert torch.equal(o3[:, 0], o4[:, 0]) and torch.equal(lse3[:, 0], lse4[:, 0])
        assert torch.equal(o3[:, 1:], o[:, 1:]) and torch.equal(lse3[:, 1:], lse[:, 1:])
        _status_ok()


# ------------------------------------------------------------------ infinite values

@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("HQ,H,K,dt", ROUTES + [(4, 4, 128, BF), (3, 1, 128, BF)])
@pytest.mark.parametrize("new,mx", [([1, 1], 1), ([5, 1, 8], 8), ([40, 1], None)])
def test_attn_infinite_values(new, mx, HQ, H, K, dt, window):
    """An infinite value is infinite in every row that sees its token, a NaN (or
    infinities of both signs) NaN, and the other rows and channels stay."""
    ctx = [100, 90, 33][:len(new)]
    x, cu, kv, table = tp._attn_inputs(HQ, H, K, K, 64, dt, new, ctx)
    kw = dict(max_new=mx, window_size=window)
    clean, _ = _attn(x, cu, kv, table, **kw)
    tol = 1e-5 if dt == F32 else 2e-2
    cases = [(ctx[0] - 10, ctx[0] - 10), (kv[0] - 1, kv[0] - 1), (ctx[0] - 3, kv[0] - 1)]
    if new[0] > 1:
        cases.append((ctx[0] + 1, ctx[0] + 2))
    pages = x["v_pages"].clone()
    for j, j2 in cases:  # tokens of request 0
        at = lambda j: (int(table[0, j // 64]), slice(None), j % 64)
        x["v_pages"][(*at(j), 3)] = math.inf
        x["v_pages"][(*at(j), 5)] = -math.inf
        x["v_pages"][(*at(j), 7)] = math.nan
        x["v_pages"][(*at(j), 9)] = math.inf
        x["v_pages"][(*at(j2), 10)] = -math.inf
        o, _ = _attn(x, cu, kv, table, **kw)
        rows = np.arange(cu[-1])
        pos = ctx[0] + rows
        sees = lambda j: torch.tensor((rows < cu[1]) & (pos >= j) & (pos - j < (window or 1 << 30)))
        s, s2 = sees(j).to(DEV), sees(j2).to(DEV)
        assert (o[s][..., 3] == math.inf).all() and (o[s][..., 5] == -math.inf).all(), (j, j2)
        assert torch.isnan(o[s][..., 7]).all() and (o[s][..., 9] == math.inf).all()
        assert (o[s2][..., 10] == -math.inf).all()
        for ch in range(K):
            seen = {3: s, 5: s, 7: s, 9: s, 10: s2}.get(ch)
            d = (o[..., ch].float() - clean[..., ch].float()).abs()
            if seen is not None:
                d = d[~seen]
            assert d.numel() == 0 or d.max() <= tol, (j, j2, ch)
        x["v_pages"].copy_(pages)
    # infinities of both signs in one channel
    j, j2 = ctx[0] - 3, kv[0] - 1
    x["v_pages"][int(table[0, j // 64]), :, j % 64, 3] = math.inf
    x["v_pages"][int(table[0, j2 // 64]), :, j2 % 64, 3] = -math.inf
    o, _ = _attn(x, cu, kv, table, **kw)
    assert torch.isnan(o[cu[1] - 1, :, 3]).all() and torch.isfinite(o[cu[1] - 1, :, 4:]).all()
    _status_ok()


# ------------------------------------------------------------- sums past the floats

def test_attn_large_values_behind_a_jump():
    """Scores that jump by 95 powers of two in a late tile over values of 2^34:
    the sums before the reference is raised pass fp32, the result does not."""
    HQ, H, K, PS, N = 16, 4, 64, 64, 40
    new, ctx = [20] * N, [700] * N
    x, _, _, _ = tp._attn_inputs(HQ, H, K, K, PS, BF, [20], [700], decay=0.0)
    cu, kv = (np.arange(N + 1) * 20).tolist(), [720] * N
    _, _, one, _, _ = tp._batch([20], [700], PS, 0)
    table = np.repeat(one, N, 0)   # every request over the same pages
    x["r_pages"].zero_()
    x["k_pages"].zero_()
    d = torch.zeros(K, device=DEV)
    d[0] = 1.0
    x["q"] = (d * 8.0).to(BF).repeat(20 * N, HQ, 1)
    x["p"] = torch.zeros(20 * N, HQ, K, device=DEV)
    for j in (300, 410):           # scale log2(e) * 8 * k = 95
        x["k_pages"][int(one[0, j // PS]), :, j % PS] = (d * (95 / 1.4427 / 8 * K ** 0.5)).to(BF)
    x["v_pages"] = (x["v_pages"].float() * 2.0 ** 34).to(BF)
    want, _ = ref.attn(x["q"][:20], x["p"][:20], [0, 20], [720], torch.tensor(one), x["k_pages"],
                       x["v_pages"], x["r_pages"], PS, K ** -0.5)
    o, _ = _attn(x, cu, kv, table)
    _status_ok()
    assert torch.isfinite(o).all()
    assert_fwd(BF, o.float() * 2.0 ** -34, np.tile(want * 2.0 ** -34, (N, 1, 1)))


# -------------------------------------------------------- pages that are none, release

def test_release_keeps_entries_that_are_no_pages_off_the_stack():
    """Table entries outside the pool are reported and dropped: the stack holds
    pages alone, in the order of the table, and a later plan opens only them."""
    PS, NP, MP = 32, 60, 60
    for bad in (-1, NP, 2 ** 31 - 1, -2 ** 31):
        tb = api.WallPagedTables(5, MP, NP, page_size=PS)
        tb.plan(_i32([40, 1, 100, 0, 32 * 40]), 40 + 1 + 100 + 32 * 40)
        _status_ok()
        held = tb.block_table.tolist()
        n_free = tb.free_count.item()
        free = tb.free_list[:n_free].tolist()
        tb.block_table[0, 1] = tb.block_table[2, 0] = tb.block_table[4, 35] = bad
        tb.release(_i32([1, 0, 1, 0, 1]))
        assert L.wall_get_status() == L.WALL_ERR_INVALID_ARG
        back = [held[0][0]] + held[2][1:4] + held[4][:35] + held[4][36:40]
        count = tb.free_count.item()
        assert tb.free_list[:count].tolist() == free + back
        assert tb.lens.tolist() == [0, 1, 0, 0, 0]
        assert (tb.block_table[[0, 2, 4]] == -1).all()
        # three pages are lost: one more than are left does not fit (nor does what
        # needs a page behind it), all that are left do
        plan = tb.plan(_i32([0, 0, 0, (count + 1) * PS, count * PS]), (2 * count + 1) * PS)
        assert plan.admitted.tolist()[3:] == [0, 0]
        plan = tb.plan(_i32([0, 0, 0, 0, count * PS]), count * PS)
        assert plan.admitted.tolist()[3:] == [1, 1]
        ids = tb.block_table[4, :count]
        assert ((ids >= 0) & (ids < NP)).all() and len(set(ids.tolist())) == count
        _status_ok()


def test_release_more_pages_than_the_pool_has():
    """Lengths that are not this stack's: reported, and the stack stays full at
    most."""
    tb = api.WallPagedTables(3, 4, 6, page_size=32)
    tb.block_table.copy_(_i32([[0, 1, 2, 3], [4, 5, 0, 1], [2, 3, 4, 5]]))
    tb.lens.fill_(128)
    tb.free_count.zero_()
    tb.release(_i32([1, 1, 1]))
    assert L.wall_get_status() == L.WALL_ERR_INVALID_ARG
    assert tb.free_count.item() == 6 and tb.free_list.tolist() == [0, 1, 2, 3, 4, 5]


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


# -------------------------------------------------- forms that other cases pass by

@pytest.mark.parametrize("HQ,H,K,V", [(1, 1, 128, 128), (4, 1, 128, 64), (6, 1, 64, 128),
                                      (8, 1, 128, 128), (4, 4, 64, 64)])
def test_attn_single_rows_do_not_see_past_their_window(HQ, H, K, V):
    """Keys and values just before the window, in the tile that it begins in,
    may be anything: the same bits."""
    ctx, window = [100, 500, 63, 31], 40
    x, cu, kv, table = tp._attn_inputs(HQ, H, K, V, 64, BF, [1] * 4, ctx)
    clean = _attn(x, cu, kv, table, max_new=1, window_size=window)
    for bad in (math.nan, math.inf, -math.inf):
        for i, n in enumerate(kv):
            for j in range(max(0, n - window - 20), n - window):
                x["v_pages"][int(table[i, j // 64]), :, j % 64] = bad
                x["k_pages"][int(table[i, j // 64]), :, j % 64] = bad
        got = _attn(x, cu, kv, table, max_new=1, window_size=window)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    _status_ok()


@pytest.mark.parametrize("hint", [False, True])
@pytest.mark.parametrize("case", [
    (4, 2, 64, 64, 64, F32, [900, 2, 411], [100, 640, 0]),
    (2, 1, 40, 24, 32, F32, [600, 1, 0, 300], [31, 7, 5, 0]),
    (3, 3, 128, 64, 128, F32, [1100, 129], [127, 0]),
    (2, 1, 64, 64, 128, F32, [40, 129, 1], [100, 0, 300]),
    (2, 2, 64, 128, 128, BF, [1000, 3], [5, 128])])
def test_append_run_by_run_in_every_form(case, hint):
    """Prompts of more than four blocks in fp32 and over pages of 128."""
    tp.test_append(case, hint)


@pytest.mark.parametrize("dt,K,signed,sink,window", [(BF, 128, True, False, 0), (BF, 64, False, True, 0),
                                                     (F32, 64, True, True, 90), (BF, 128, True, True, 50)])
def test_serving_run_with_sink_and_signed_gates(dt, K, signed, sink, window):
    """A prompt, single tokens, drafts and a chunk of one request, beside
    another: every row equals the oracle's forward of the whole sequence."""
    HQ, H, PS = 4, 2, 64
    gen = torch.Generator().manual_seed(17)
    lens = [260, 150]
    sk = torch.randn(HQ, generator=gen) if sink else None
    seqs = []
    for n in lens:
        g = tp._rand(gen, n, HQ, K, dtype=dt, amp=0.04)
        seqs.append(dict(q=tp._rand(gen, n, HQ, K, dtype=dt), k=tp._rand(gen, n, H, K, dtype=dt),
                         v=tp._rand(gen, n, H, K, dtype=dt), g=g if signed else -g.abs()))
    want = [wo.forward(*(s[n][None].cpu() for n in "qkvg"), scale=K ** -0.5, sink_bias=sk,
                       window_size=window or None)[0][0] for s in seqs]
    tb = api.WallPagedTables(2, 5, 10, page_size=PS)
    cache = api.WallPagedCache(tb, H, HQ, K, K, dtype=dt, window_size=window or None,
                               sink_bias=None if sk is None else sk.to(DEV))
    at = [0, 0]
    for new in ([130, 1], [1, 60], [1, 1], [8, 3], [60, 1], [1, 84], [59, 0]):
        cat = {x: torch.cat([s[x][a:a + n] for s, a, n in zip(seqs, at, new)]) for x in "qkvg"}
        o = cache.step(tb.plan(_i32(new), sum(new)), cat["q"], cat["k"], cat["v"], cat["g"],
                       max_new=max(new))
        r0 = 0
        for i, n in enumerate(new):
            assert_fwd(dt, o[r0:r0 + n], want[i][at[i]:at[i] + n], what=f"request {i}")
            at[i] += n
            r0 += n
    assert at == lens
    _status_ok()
