"""GPU tests of the paged cache: the page plan, the append, the attention and
the three in a row, against 64-bit request-by-request references and the
framework's fp64 oracle, at the lengths, masks and pages where they can go
wrong."""
import random

import numpy as np
import pytest
import torch

from channel_decay_softmax_b200 import _lib as L
from channel_decay_softmax_b200 import api
from oracle import wall_oracle as wo
from tests import paged_reference as ref
from tests.helpers import assert_fwd, max_abs

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _status_ok():
    assert L.wall_get_status() == L.WALL_OK


# ---------------------------------------------------------------------- plan

def _plan_ref(new, lens, table, free, count, PS, T):
    """The definition, request by request."""
    N, MP = table.shape
    table, lens_out = table.copy(), list(lens)
    cu, kv, adm = [0], [], []
    slots = np.full(T, -1, np.int64)
    need_sum, used = 0, 0
    for i in range(N):
        n = max(new[i], 0)
        rows = cu[-1] + n
        held, want = -(-lens[i] // PS), -(-(lens[i] + n) // PS)
        fits = want <= MP and rows <= T
        need = want - held if fits else 0
        need_sum += need
        ok = fits and (need == 0 or need_sum <= count)
        if ok and need:
            for x in range(need):
                table[i, held + x] = free[count - 1 - (need_sum - need + x)]
            used = need_sum
        if ok:
            for x in range(n):
                pos = lens[i] + x
                slots[cu[-1] + x] = int(table[i, pos // PS]) * PS + pos % PS
            lens_out[i] = lens[i] + n
        cu.append(min(rows, T))
        kv.append(lens[i] + n if ok else 0)
        adm.append(int(ok))
    return cu, kv, slots, adm, table, lens_out, count - used


def _tables_with(ctx, PS, MP, NP, seed, spare_table=None):
    """A table whose requests hold the pages of ctx tokens, and the rest free."""
    rng = np.random.default_rng(seed)
    perm = rng.permutation(NP).astype(np.int32)
    table = np.full((len(ctx), MP), -1, np.int32)
    at = 0
    for i, c in enumerate(ctx):
        h = -(-c // PS)
        table[i, :h] = perm[at:at + h]
        at += h
    free = np.full(NP, -1, np.int32)
    free[:NP - at] = perm[at:]
    return table, free, NP - at


@pytest.mark.parametrize("N,new_hi,ctx_hi,PS,pages,rows", [
    (1, 1, 0, 32, "plenty", "exact"), (1, 700, 500, 64, "plenty", "padded"),
    (5, 40, 300, 32, "plenty", "exact"), (33, 3, 900, 128, "plenty", "padded"),
    (64, 200, 100, 32, "short", "exact"), (64, 200, 100, 32, "plenty", "short"),
    (1023, 9, 400, 64, "short", "padded"), (1025, 9, 400, 64, "plenty", "exact"),
    (3000, 30, 600, 32, "plenty", "exact"), (2500, 2, 100, 32, "none", "padded")])
def test_plan(N, new_hi, ctx_hi, PS, pages, rows):
    rng = random.Random(N * 7 + PS)
    ctx = [rng.randint(0, ctx_hi) for _ in range(N)]
    new = [rng.randint(0, new_hi) for _ in range(N)]
    held = sum(-(-c // PS) for c in ctx)
    want = sum(-(-(c + n) // PS) for c, n in zip(ctx, new))
    MP = max(1, -(-(ctx_hi + new_hi) // PS) - (1 if rows == "short" else 0))
    MP = max(MP, max(-(-c // PS) for c in ctx))
    NP = max(1, {"plenty": want + 5, "short": held + (want - held) // 2, "none": held}[pages])
    total = sum(new)
    T = {"exact": total, "padded": total + 37, "short": total * 2 // 3}[rows]
    table, free, count = _tables_with(ctx, PS, MP, NP, seed=N)
    cu, kv, slots, adm, table_w, lens_w, count_w = _plan_ref(new, ctx, table, free, count, PS, T)
    for in_place in (False, True):
        lens, cnt, tb = _i32(ctx), _i32([count]), _i32(table)
        lo = lens if in_place else torch.empty_like(lens)
        co = cnt if in_place else torch.empty_like(cnt)
        pl = api.wall_paged_plan(_i32(new), lens, tb, _i32(free), cnt, PS, T,
                                 lens_out=None if in_place else lo,
                                 free_count_out=None if in_place else co)
        assert pl.cu_q.tolist() == cu
        assert pl.kv_lens.tolist() == kv
        assert pl.admitted.tolist() == adm
        assert np.array_equal(pl.slot_map.cpu().numpy(), slots)
        assert np.array_equal(tb.cpu().numpy(), table_w)
        assert lo.tolist() == lens_w and co.item() == count_w
        if not in_place:
            assert lens.tolist() == ctx and cnt.item() == count
    _status_ok()


def test_plan_records_a_bad_stack_and_negative_lengths():
    """A free count beyond the pool or a negative length is reported, and no
    entry outside the stack is read."""
    table, free, count = _tables_with([10, 40], 32, 4, 8, seed=1)
    api.wall_paged_plan(_i32([1, 1]), _i32([10, 40]), _i32(table), _i32(free), _i32([9]), 32, 2)
    assert L.wall_get_status() == L.WALL_ERR_INVALID_ARG
    pl = api.wall_paged_plan(_i32([-5, 1]), _i32([10, 40]), _i32(table), _i32(free),
                             _i32([count]), 32, 2)
    assert L.wall_get_status() == L.WALL_ERR_INVALID_ARG
    assert pl.cu_q.tolist() == [0, 0, 1]


def test_release_and_reuse():
    """Pages of finished requests go back and are opened again; nothing is lost
    or doubled over a long run of plans and releases."""
    PS, N, MP, NP = 32, 40, 6, 150
    tb = api.WallPagedTables(N, MP, NP, page_size=PS)
    rng = random.Random(3)
    lens = [0] * N
    for step in range(25):
        new = [rng.choice([0, 1, 1, rng.randint(0, 60)]) for _ in range(N)]
        pl = tb.plan(_i32(new), sum(new))
        for i, a in enumerate(pl.admitted.tolist()):
            lens[i] += new[i] if a else 0
        assert tb.lens.tolist() == lens
        held = tb.block_table[tb.block_table >= 0].tolist()
        free = tb.free_list[:tb.free_count.item()].tolist()
        assert sorted(held + free) == list(range(NP))
        fin = [int(rng.random() < 0.15 or x >= MP * PS - 60) for x in lens]
        tb.release(_i32(fin))
        lens = [0 if f else x for f, x in zip(fin, lens)]
        assert tb.lens.tolist() == lens
        assert all((tb.block_table[i] == -1).all() for i, f in enumerate(fin) if f)
    _status_ok()


# -------------------------------------------------------------------- append

def _rand(gen, *shape, dtype=BF, amp=1.0):
    return (torch.randn(*shape, generator=gen) * amp).to(dtype).to(DEV)


def _batch(new, ctx, PS, seed, extra_rows=0, refused=()):
    """Plan arrays of a batch whose pages are all opened (host-made)."""
    kv = [0 if i in refused else c + n for i, (c, n) in enumerate(zip(ctx, new))]
    MP = max(1, max(-(-(c + n) // PS) for c, n in zip(ctx, new)))
    NP = sum(-(-(c + n) // PS) for c, n in zip(ctx, new)) + 2
    table, _, _ = _tables_with([c + n for c, n in zip(ctx, new)], PS, MP, NP, seed)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    slots = np.full(cu[-1] + extra_rows, -1, np.int64)
    for i, (c, n) in enumerate(zip(ctx, new)):
        if kv[i]:
            pos = c + np.arange(n)
            slots[cu[i]:cu[i + 1]] = table[i, pos // PS].astype(np.int64) * PS + pos % PS
    return cu, kv, table, slots, NP


APPEND = [
    # HQ, H, K, V, PS, dtype, new, ctx
    (4, 2, 64, 64, 64, BF, [1, 1, 1], [0, 64, 63]),
    (4, 4, 128, 128, 32, BF, [70, 1, 33, 5], [0, 31, 95, 500]),
    (3, 1, 128, 64, 64, BF, [200, 0, 63, 1], [1, 7, 0, 64]),
    (2, 2, 64, 128, 128, BF, [129, 300], [127, 0]),
    (6, 3, 64, 64, 32, F32, [40, 1, 2, 64], [0, 5, 32, 30]),
    (5, 5, 40, 24, 64, F32, [3, 130], [62, 1]),
    (2, 1, 8, 8, 128, BF, [260], [130]),
    (16, 4, 128, 128, 64, BF, [900, 2, 411], [100, 640, 0]),
]


def _append_inputs(case, seed=0, amp=0.02, extra_rows=0, refused=()):
    HQ, H, K, V, PS, dt, new, ctx = case
    gen = torch.Generator().manual_seed(100 + seed)
    cu, kv, table, slots, NP = _batch(new, ctx, PS, seed, extra_rows, refused)
    T = cu[-1] + extra_rows
    x = dict(k=_rand(gen, T, H, K, dtype=dt), v=_rand(gen, T, H, V, dtype=dt),
             g=-_rand(gen, T, HQ, K, dtype=dt, amp=amp).abs())
    pools = dict(k_pages=_rand(gen, NP, HQ, PS, K, dtype=dt),
                 v_pages=_rand(gen, NP, H, PS, V, dtype=dt),
                 r_pages=torch.randint(-40, 0, (NP, HQ, K), generator=gen).to(torch.int32).to(DEV))
    # the prefix at the last cached token: within a page's reach of its anchor
    carry = torch.randint(-(9 << 24), 0, (len(new), HQ, K), generator=gen, dtype=torch.int64).to(DEV)
    for i, c in enumerate(ctx):
        if c > 0:
            carry[i] += pools["r_pages"][int(table[i, (c - 1) // PS])].long() << 24
    return x, pools, carry, cu, kv, table, slots


@pytest.mark.parametrize("case", APPEND)
@pytest.mark.parametrize("hint", [False, True])
def test_append(case, hint):
    HQ, H, K, V, PS, dt, new, ctx = case
    x, pools, carry, cu, kv, table, slots = _append_inputs(case)
    want = ref.append(x["k"], x["v"], x["g"], cu, kv, torch.tensor(slots), carry=carry, PS=PS,
                      **pools)
    out = torch.full_like(carry, 77)
    p = api.wall_paged_append(x["k"], x["v"], x["g"], _i32(cu), _i32(kv),
                              torch.tensor(slots, device=DEV), carry=carry, carry_out=out,
                              max_new=max(new) if hint else None, **pools)
    _status_ok()
    # whole numbers: exact
    assert np.array_equal(out.cpu().numpy(), want[4])
    assert np.array_equal(pools["r_pages"].cpu().numpy(), want[3])
    # p: one rounding of an exact number; the value rows: copied
    got_p = ref.f64(p)
    assert np.all(np.abs(got_p - want[0]) <= 2.0 ** -24 * np.abs(want[0]))
    assert np.array_equal(ref.f64(pools["v_pages"]), want[2])
    # the key rows: p's rounding (|p| ln 2 2^-24), the exponential's 2^-22 and
    # the product's 2^-24, then half a step of the type
    half = torch.finfo(dt).eps / 2
    reach = float(np.nanmax(np.abs(want[0])))
    rel = half * 1.01 + (reach * 0.7 + 6) * 2.0 ** -24
    assert np.all(np.abs(ref.f64(pools["k_pages"]) - want[1]) <= rel * np.abs(want[1]))


def test_append_in_pieces_leaves_the_same_bits():
    """One call, chunks that end inside pages, token by token: the pools, the
    anchors, p and the carry agree bit for bit; carry in place."""
    HQ, H, K, V, PS, Ttot = 4, 2, 128, 128, 64, 333
    gen = torch.Generator().manual_seed(8)
    k, v = _rand(gen, Ttot, H, K), _rand(gen, Ttot, H, V)
    g = -_rand(gen, Ttot, HQ, K, amp=0.1).abs()
    outs = []
    for cuts in ([Ttot], [1] * 70 + [Ttot - 70], [63, 2, 100, 128, 40]):
        tb = api.WallPagedTables(2, 6, 9, page_size=PS)
        c = api.WallPagedCache(tb, H, HQ, K, V)
        for t in (c.k_pages, c.v_pages, c.r_pages, c.carry):
            t.zero_()
        ps, at = [], 0
        for n in cuts:
            pl = tb.plan(_i32([0, n]), n)
            ps.append(c.append(pl, k[at:at + n], v[at:at + n], g[at:at + n],
                               max_new=n if n < 5 else None))
            at += n
        outs.append((torch.cat(ps), c.k_pages, c.v_pages, c.r_pages, c.carry))
    _status_ok()
    for got in outs[1:]:
        for a, b in zip(outs[0], got):
            assert torch.equal(a, b)


def test_append_skips_refused_and_padded_rows():
    case = (4, 2, 64, 64, 32, BF, [5, 40, 1, 3], [30, 0, 64, 10])
    x, pools, carry, cu, kv, table, slots = _append_inputs(case, extra_rows=9, refused=(1, 2))
    for n in ("k", "v", "g"):  # rows that nothing may read into a result
        x[n][cu[1]:cu[3]] = float("nan")
        x[n][cu[-1]:] = float("nan")
    want = ref.append(x["k"], x["v"], x["g"], cu, kv, torch.tensor(slots), carry=carry, PS=32, **pools)
    before = carry.clone()
    api.wall_paged_append(x["k"], x["v"], x["g"], _i32(cu), _i32(kv),
                          torch.tensor(slots, device=DEV), carry=carry, **pools)
    _status_ok()
    assert np.array_equal(carry.cpu().numpy(), want[4])
    assert torch.equal(carry[1:3], before[1:3])
    assert torch.isfinite(pools["k_pages"]).all() and torch.isfinite(pools["v_pages"]).all()
    assert np.array_equal(ref.f64(pools["v_pages"]), want[2])


def test_append_special_gates():
    """A NaN gate marks its own token and no other; a gate of -inf at a page's
    start is a hard reset; inside a page it leaves the page's range, which is
    reported; a slot outside the pool is reported and not followed."""
    HQ, H, K, PS = 2, 1, 64, 32
    def call(g, slots=None, n=40):
        pools = dict(k_pages=torch.zeros(4, HQ, PS, K, dtype=F32, device=DEV),
                     v_pages=torch.zeros(4, H, PS, K, dtype=F32, device=DEV),
                     r_pages=torch.zeros(4, HQ, K, dtype=torch.int32, device=DEV))
        carry = torch.zeros(1, HQ, K, dtype=torch.int64, device=DEV)
        slots = torch.arange(n, device=DEV) if slots is None else slots
        one = torch.ones(n, H, K, device=DEV)
        p = api.wall_paged_append(one, one, g, _i32([0, n]), _i32([n]), slots, carry=carry, **pools)
        return p, pools, carry
    g = torch.zeros(40, HQ, K, device=DEV)
    g[7, 1, 5] = float("nan")
    p, pools, carry = call(g)
    _status_ok()
    bad = torch.isnan(p)
    assert bad.sum() == 1 and bad[7, 1, 5]
    bad = torch.isnan(pools["k_pages"])
    assert bad.sum() == 1 and bad[0, 1, 7, 5]
    g = torch.zeros(40, HQ, K, device=DEV)
    g[32] = float("-inf")
    p, pools, carry = call(g)
    _status_ok()
    assert (pools["r_pages"][1] == -128).all() and (p == 0).all()
    assert (carry == -(1 << 31)).all()
    g[20, 0, 0] = float("-inf")
    call(g)
    assert L.wall_get_status() == L.WALL_ERR_RANGE
    # the same as the only new token of a call: the range is left in one step
    # that passes 32 bits, too
    for first in (0.0, -50.0):
        pools = dict(k_pages=torch.zeros(2, HQ, PS, K, dtype=F32, device=DEV),
                     v_pages=torch.zeros(2, H, PS, K, dtype=F32, device=DEV),
                     r_pages=torch.zeros(2, HQ, K, dtype=torch.int32, device=DEV))
        carry = torch.zeros(1, HQ, K, dtype=torch.int64, device=DEV)
        one = torch.ones(1, H, K, device=DEV)
        for n, step in enumerate((0.0, first, float("-inf"))):
            assert L.wall_get_status() == L.WALL_OK
            api.wall_paged_append(one, one, torch.full((1, HQ, K), step, device=DEV), _i32([0, 1]),
                                  _i32([n + 1]), torch.tensor([n], device=DEV), carry=carry,
                                  max_new=1, **pools)
        assert L.wall_get_status() == L.WALL_ERR_RANGE
    slots = torch.arange(40, device=DEV)
    slots[3], slots[35] = -1, 4 * PS
    p, pools, carry = call(torch.zeros(40, HQ, K, device=DEV), slots)
    assert L.wall_get_status() == L.WALL_ERR_INVALID_ARG
    assert (pools["v_pages"].sum() == 38 * H * K).item()


# ------------------------------------------------------------------ attention

def _attn_inputs(HQ, H, K, V, PS, dt, new, ctx, seed=0, extra_rows=0, refused=(), decay=0.03):
    gen = torch.Generator().manual_seed(300 + seed)
    cu, kv, table, slots, NP = _batch(new, ctx, PS, seed, extra_rows, refused)
    T = cu[-1] + extra_rows
    tilt = 0.5 + torch.rand(HQ, K, generator=gen)
    grow = torch.exp2(decay * torch.arange(PS).float()[:, None] * tilt[:, None, :])
    x = dict(k_pages=(torch.randn(NP, HQ, PS, K, generator=gen) * grow).to(dt).to(DEV),
             v_pages=_rand(gen, NP, H, PS, V, dtype=dt))
    r = torch.zeros(NP, HQ, K, dtype=torch.int32)
    pos = np.zeros(T, np.int64)
    for i in range(len(new)):
        for j in range(table.shape[1]):
            if table[i, j] >= 0:
                r[int(table[i, j])] = torch.floor(-decay * PS * j * tilt + 0.5).int()
        pos[cu[i]:cu[i + 1]] = ctx[i] + np.arange(new[i])
    x["r_pages"] = r.to(DEV)
    x["q"] = _rand(gen, T, HQ, K, dtype=dt)
    x["p"] = (-decay * torch.tensor(pos % PS).float()[:, None, None] * tilt
              - 0.3 * torch.rand(T, HQ, K, generator=gen)).to(DEV)
    return x, cu, kv, table


def _attn_case(HQ, H, K, V, PS, dt, new, ctx, window=0, sink=False, hint=False, seed=0,
               extra_rows=0, refused=(), poison=False, decay=0.03):
    x, cu, kv, table = _attn_inputs(HQ, H, K, V, PS, dt, new, ctx, seed, extra_rows, refused, decay)
    sk = torch.randn(HQ, generator=torch.Generator().manual_seed(5)).to(DEV) if sink else None
    scale = K ** -0.5
    o_ref, lse_ref = ref.attn(x["q"], x["p"], cu, kv, torch.tensor(table), x["k_pages"],
                              x["v_pages"], x["r_pages"], PS, scale, sk, window)
    if poison:  # cached rows past the last token, and pages nobody holds
        held = np.zeros((x["k_pages"].shape[0], PS), bool)
        for i, n in enumerate(kv):
            for j in range(n):
                held[table[i, j // PS], j % PS] = True
        gone = torch.tensor(~held, device=DEV)
        x["k_pages"].masked_fill_(gone[:, None, :, None], float("nan"))
        x["v_pages"].masked_fill_(gone[:, None, :, None], float("nan"))
    o, lse = api.wall_paged_attn(x["q"], x["p"], _i32(cu), _i32(kv), _i32(table), x["k_pages"],
                                 x["v_pages"], x["r_pages"], max_new=max(new) if hint else None,
                                 scale=scale, sink_bias=sk, window_size=window, return_lse=True)
    _status_ok()
    n = cu[-1]
    empty = np.isinf(lse_ref[:n])
    assert np.array_equal(np.isinf(ref.f64(lse[:n])), empty)
    assert_fwd(dt, o[:n], o_ref[:n], what="paged")
    e = max_abs(lse[:n], lse_ref[:n], ~empty)
    assert e <= (1e-5 if dt == F32 else 2e-2), e
    return x, o, lse


SHAPES = [(4, 2, 64, 64, BF), (2, 2, 128, 128, BF), (8, 1, 128, 128, BF), (3, 3, 128, 64, BF),
          (2, 1, 64, 128, BF), (4, 2, 64, 64, F32), (3, 1, 40, 24, F32), (12, 1, 64, 64, BF),
          (2, 2, 24, 40, BF)]


@pytest.mark.parametrize("HQ,H,K,V,dt", SHAPES)
@pytest.mark.parametrize("PS", [32, 64, 128])
def test_attn_decode(HQ, H, K, V, dt, PS):
    """One token a request: empty, page-sized and ragged contexts."""
    _attn_case(HQ, H, K, V, PS, dt, [1] * 7, [0, 1, 31, 63, 64, 127, 300], hint=True,
               sink=PS == 64, poison=True)


@pytest.mark.parametrize("HQ,H,K,V,dt", SHAPES + [(5, 1, 128, 128, BF), (1, 1, 64, 64, BF)])
@pytest.mark.parametrize("PS,window", [(32, 0), (64, 0), (128, 0), (64, 1), (32, 5), (128, 70)])
def test_attn_few_rows(HQ, H, K, V, dt, PS, window):
    """At most eight tokens a request, and that many announced: rows on both
    sides of a page's and a tile's end, windows that end between them."""
    _attn_case(HQ, H, K, V, PS, dt, [8, 2, 1, 0, 5, 3, 8, 7, 2], [0, 31, 64, 9, 60, 127, 249, 500, 0],
               window=window, sink=window == 5, hint=True, poison=True)


@pytest.mark.parametrize("window", [0, 4])
def test_attn_few_rows_masked_values_may_be_nan(window):
    """A value that is not finite reaches the rows that see its token alone."""
    new, ctx, HQ, H, K = [6, 8], [90, 28], 4, 2, 128
    x, cu, kv, table, = _attn_inputs(HQ, H, K, K, 64, BF, new, ctx)
    call = lambda: api.wall_paged_attn(x["q"], x["p"], _i32(cu), _i32(kv), _i32(table), x["k_pages"],
                                       x["v_pages"], x["r_pages"], window_size=window, max_new=8)
    clean = call()
    for bad in (float("nan"), float("inf")):
        pages = x["v_pages"].clone()
        for i, row in ((0, 3), (1, 5)):  # the request's token `row`
            j = ctx[i] + row
            x["v_pages"][int(table[i, j // 64]), :, j % 64] = bad
        o = call()
        for i, row in ((0, 3), (1, 5)):
            for t in range(new[i]):
                sees = t >= row and (window == 0 or t - row < window)
                mine = o[cu[i] + t]
                assert not torch.isfinite(mine).any() if sees else torch.equal(mine, clean[cu[i] + t]), (i, t)
        x["v_pages"] = pages
    _status_ok()


@pytest.mark.parametrize("sink", [False, True])
def test_attn_few_rows_refused_and_padded(sink):
    _attn_case(4, 2, 128, 128, 64, BF, [1, 8, 3, 5], [70, 0, 60, 2], sink=sink, refused=(1, 2),
               extra_rows=5, hint=True)


def test_attn_few_rows_are_repeatable_captured_and_on_two_streams():
    """Units cut over many CTAs: the same bits from repeated calls, from two
    streams at once and from a graph, whose lengths change under it."""
    new, ctx = [8, 1, 5, 2], [6000, 300, 2500, 64]
    x, cu, kv, table = _attn_inputs(4, 1, 128, 128, 64, BF, new, ctx, decay=0.002)
    cu_t, kv_t, tb = _i32(cu), _i32(kv), _i32(table)
    call = lambda: api.wall_paged_attn(x["q"], x["p"], cu_t, kv_t, tb, x["k_pages"], x["v_pages"],
                                       x["r_pages"], max_new=8, return_lse=True)
    first = call()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(call())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(first, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    kv_t.copy_(_i32([n - 3 if n > 20 else n for n in kv]))
    want = call()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, out)) and not torch.equal(want[0], first[0])
    _status_ok()


@pytest.mark.parametrize("decay", [0.0, 0.6, 2.0])
def test_attn_few_rows_decay(decay):
    """Gates from none to ones that forget a page within a page: prefixes of up
    to 2.0 * 31 * 1.5 = 93 powers of two, of the 100 that a page may hold."""
    PS = 32
    _attn_case(4, 1, 128, 128, PS, BF, [8, 4, 2], [200, 30, 95], hint=True, decay=decay)


@pytest.mark.parametrize("HQ,H", [(1, 1), (2, 1), (4, 1), (8, 2)])
def test_attn_decode_keeps_its_order_of_tiles(HQ, H):
    """Requests of one tile between requests of many, over and over: warps that
    have no tile of a request must not run ahead of those that have, and every
    run gives the same bits."""
    ctx = [int(c) for c in np.random.default_rng(HQ).choice([0, 20, 70, 250, 500, 1500], 240)]
    x, o, lse = _attn_case(HQ, H, 128, 128, 64, BF, [1] * len(ctx), ctx, hint=True)
    cu, kv, table, _, _ = _batch([1] * len(ctx), ctx, 64, 0)
    for _ in range(30):
        again = api.wall_paged_attn(x["q"], x["p"], _i32(cu), _i32(kv), _i32(table), x["k_pages"],
                                    x["v_pages"], x["r_pages"], max_new=1, scale=128 ** -0.5)
        assert torch.equal(again, o)
    _status_ok()


@pytest.mark.parametrize("HQ,H,K,V,dt", SHAPES)
@pytest.mark.parametrize("new,ctx", [
    ([2, 5], [0, 100]), ([33, 1, 64], [0, 40, 95]), ([129], [0]), ([40, 128, 1, 0, 130], [90, 128, 200, 7, 1])])
def test_attn_chunks(HQ, H, K, V, dt, new, ctx):
    """Chunks beside single tokens, over cached contexts of any alignment."""
    _attn_case(HQ, H, K, V, 64, dt, new, ctx, sink=new[0] == 33, poison=True)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("PS", [32, 128])
@pytest.mark.parametrize("window", [1, 2, 31, 64, 129, 200])
def test_attn_window(dt, PS, window):
    _attn_case(4, 2, 64, 64, PS, dt, [1, 140, 3], [260, 130, 64], window=window, sink=window == 64,
               poison=True)


@pytest.mark.parametrize("K,dt", [(128, BF), (64, BF), (64, F32)])
def test_attn_refused_and_padded_rows(K, dt):
    """Refused requests' rows are empty (the sink's bias with a sink), whatever
    their p holds; rows past the last request stay as they were."""
    for sink in (False, True):
        _attn_case(4, 2, K, K, 64, dt, [1, 20, 1, 150], [70, 0, 3, 2], sink=sink,
                   refused=(1, 2), extra_rows=5)
    x, cu, kv, table = _attn_inputs(4, 2, K, K, 64, dt, [1, 20, 1, 3], [70, 0, 3, 2], 0, 5, (1, 2))
    x["p"][cu[1]:cu[3]] = float("nan")
    x["p"][cu[-1]:] = float("nan")
    x["q"][cu[-1]:] = float("nan")
    o = torch.full((cu[-1] + 5, 4, K), 7.0, dtype=dt, device=DEV)
    ws = torch.empty(L.wall_paged_attn_workspace(dt, 4, cu[-1] + 5, 0, 2, 4, K, K),
                     dtype=torch.uint8, device=DEV)
    L.wall_paged_attn(x["q"], x["p"], _i32(cu), _i32(kv), _i32(table), 4, cu[-1] + 5, 0,
                      table.shape[1], 2, 4, K, K, 64, x["k_pages"].shape[0], x["k_pages"],
                      x["v_pages"], x["r_pages"], None, 0.0, 0, o, None, ws)
    _status_ok()
    assert (o[cu[-1]:] == 7).all() and (o[cu[1]:cu[3]] == 0).all()
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("new", [[1, 1], [60, 1], [200, 130]])
@pytest.mark.parametrize("K,dt", [(128, BF), (64, F32)])
def test_attn_masked_values_may_be_nan(new, K, dt):
    """A NaN in a token's value (and key) row reaches the rows that see the
    token and no other: not the earlier rows of the same chunk, not rows whose
    window has passed it, not another request."""
    ctx, window = [100, 50], 40
    x, cu, kv, table = _attn_inputs(2, 1, K, K, 64, dt, new, ctx)
    args = lambda: (x["q"], x["p"], _i32(cu), _i32(kv), _i32(table), x["k_pages"], x["v_pages"],
                    x["r_pages"])
    clean = api.wall_paged_attn(*args(), window_size=window)
    j = kv[0] - max(1, new[0] // 2)  # a token of request 0
    x["v_pages"][int(table[0, j // 64]), :, j % 64] = float("nan")
    x["k_pages"][int(table[0, j // 64]), :, j % 64] = float("nan")
    got = api.wall_paged_attn(*args(), window_size=window)
    pos = np.concatenate([c + np.arange(n) for c, n in zip(ctx, new)])
    sees = (pos >= j) & (pos - j < window) & (np.arange(cu[-1]) < cu[1])
    sees = torch.tensor(sees, device=DEV)
    assert torch.isnan(got[sees]).all()
    # the other rows: their values up to what the general kernel differs by
    assert torch.isfinite(got[~sees]).all()
    assert max_abs(got[~sees], clean[~sees]) <= (1e-5 if dt == F32 else 2e-2)
    _status_ok()


def test_attn_long_context_and_many_splits():
    """One request over many CTAs, and many requests over few."""
    _attn_case(2, 1, 128, 128, 64, BF, [1], [5000], hint=True)
    _attn_case(2, 2, 64, 64, 32, BF, [2], [3000])
    _attn_case(2, 1, 64, 64, 32, F32, [1], [2500], hint=True)
    _attn_case(1, 1, 64, 64, 32, BF, [1] * 700, [i % 90 for i in range(700)], hint=True)
    _attn_case(1, 1, 64, 64, 32, BF, [1 + i % 3 for i in range(400)], [i % 70 for i in range(400)])


@pytest.mark.parametrize("K,window", [(128, 130), (64, 0), (128, 0)])
def test_attn_many_units(K, window):
    """More units than CTAs, of one to three tiles each: every CTA's pipeline
    runs across units, with and without whole ones in its share."""
    new = [2 + (37 * i) % 140 for i in range(120)]
    _attn_case(2, 1, K, K, 64, BF, new, [(53 * i) % 200 for i in range(120)], window=window,
               poison=True)


def test_attn_long_windowed_prompts():
    """Many tiles and many units a CTA, two partly masked tiles in each."""
    _attn_case(16, 2, 128, 128, 64, BF, [520, 390], [700, 30], window=300, sink=True)


@pytest.mark.parametrize("K,dt", [(128, BF), (64, BF), (64, F32)])
@pytest.mark.parametrize("decay", [1.2, 2.0])
def test_attn_strong_decay(K, dt, decay):
    """Channels that lose over a power of two a token: exponents far beyond
    what one anchor of a row block spans."""
    _attn_case(2, 1, K, K, 32, dt, [1, 150, 40], [90, 70, 0], decay=decay)


@pytest.mark.parametrize("jump", [20.0, 300.0])
def test_attn_scores_that_jump(jump):
    """Scores that rise from tile to tile by far more than one reference serves
    (300 units of log2: past what fp32 sums hold against it), and keys that
    take the whole weight."""
    x, cu, kv, table = _attn_inputs(2, 1, 128, 128, 64, BF, [150, 2], [500, 300], decay=0.0)
    x["p"].zero_()
    x["r_pages"].zero_()
    for i, n in enumerate(kv):
        for j in (60, 200, 330, 420, 610):
            if j < n:
                page, off = int(table[i, j // 64]), j % 64
                # along the first query row: a score of about `jump` times its rank
                d = x["q"][cu[i]].float()
                x["k_pages"][page, :, off] = (d * (jump * j / 200.0 / 1.4427 / (128 ** -0.5))
                                              / (d * d).sum(-1, keepdim=True)).to(BF)
    o_ref, _ = ref.attn(x["q"], x["p"], cu, kv, torch.tensor(table), x["k_pages"], x["v_pages"],
                        x["r_pages"], 64, 128 ** -0.5)
    o = api.wall_paged_attn(x["q"], x["p"], _i32(cu), _i32(kv), _i32(table), x["k_pages"],
                            x["v_pages"], x["r_pages"])
    _status_ok()
    assert_fwd(BF, o, o_ref)


def test_attn_far_positions_are_exact():
    """Prefixes of millions of powers of two: only differences matter, to the
    last bit."""
    x, cu, kv, table = _attn_inputs(2, 1, 64, 64, 64, BF, [1, 70], [200, 100])
    args = lambda: (x["q"], x["p"], _i32(cu), _i32(kv), _i32(table), x["k_pages"], x["v_pages"],
                    x["r_pages"])
    near = api.wall_paged_attn(*args())
    x["r_pages"] -= 50_000_000
    assert torch.equal(near, api.wall_paged_attn(*args()))
    _status_ok()


def test_attn_reports_bad_pages_and_bounds():
    """A page id outside the pool, and more rows than max_new, are reported."""
    x, cu, kv, table = _attn_inputs(2, 1, 64, 64, 64, BF, [1, 40], [200, 100])
    call = lambda tb, mx=None: api.wall_paged_attn(
        x["q"], x["p"], _i32(cu), _i32(kv), _i32(tb), x["k_pages"], x["v_pages"], x["r_pages"],
        max_new=mx)
    for bad in (-1, x["k_pages"].shape[0], 2 ** 31 - 1):
        for i, j in ((0, 1), (1, 0), (1, 2)):
            t2 = table.copy()
            t2[i, j] = bad
            call(t2)
            assert L.wall_get_status() == L.WALL_ERR_INVALID_ARG, (bad, i, j)
    call(table, 39)
    assert L.wall_get_status() == L.WALL_ERR_INVALID_ARG
    # a table narrower than the lengths
    call(np.ascontiguousarray(table[:, :2]))
    assert L.wall_get_status() == L.WALL_ERR_INVALID_ARG
    call(table)
    _status_ok()


@pytest.mark.parametrize("HQ,H,K,dt", [(2, 1, 64, BF), (12, 1, 64, BF), (2, 1, 64, F32)])
@pytest.mark.parametrize("new,mx", [([1, 1], 1), ([1, 5], 8), ([1, 40], None), ([40, 3], None)])
def test_attn_lengths_past_the_table_are_refused(HQ, H, K, dt, new, mx):
    """A length beyond what the block table holds (up to the largest int) is
    reported, costs nothing and leaves the other requests as they are."""
    x, cu, kv, table = _attn_inputs(HQ, H, K, K, 64, dt, new, [100, 200])
    call = lambda lens: api.wall_paged_attn(x["q"], x["p"], _i32(cu), _i32(lens), _i32(table),
                                            x["k_pages"], x["v_pages"], x["r_pages"], max_new=mx)
    want = call(kv)
    _status_ok()
    for far in (table.shape[1] * 64 + 1, 2 ** 31 - 1):
        o = call([kv[0], far])
        assert L.wall_get_status() == L.WALL_ERR_INVALID_ARG
        assert (o[cu[1]:] == 0).all()
        assert (o[:cu[1]] - want[:cu[1]]).abs().max() <= 2e-2  # another division of the work


@pytest.mark.parametrize("new,mx", [([1], 1), ([5], None), ([700], None)])
def test_append_lengths_of_the_largest_int_are_refused(new, mx):
    HQ, H, K, PS = 2, 1, 64, 64
    pools = dict(k_pages=torch.zeros(16, HQ, PS, K, dtype=BF, device=DEV),
                 v_pages=torch.zeros(16, H, PS, K, dtype=BF, device=DEV),
                 r_pages=torch.zeros(16, HQ, K, dtype=torch.int32, device=DEV))
    T = new[0]
    one = torch.ones(T, H, K, dtype=BF, device=DEV)
    for far in (2 ** 31 - 1, 2 ** 31 - 100):
        carry = torch.full((1, HQ, K), 7, dtype=torch.int64, device=DEV)
        api.wall_paged_append(one, one, torch.ones(T, HQ, K, dtype=BF, device=DEV), _i32([0, T]),
                              _i32([far]), torch.arange(T, device=DEV), carry=carry, max_new=mx, **pools)
        _status_ok()
        assert (carry == 7).all() and all((t == 0).all() for t in pools.values())


def test_attn_pages_before_the_window_may_be_gone():
    x, cu, kv, table = _attn_inputs(4, 2, 128, 128, 32, BF, [1, 130], [300, 290])
    args = lambda tb: (x["q"], x["p"], _i32(cu), _i32(kv), _i32(tb), x["k_pages"], x["v_pages"],
                       x["r_pages"])
    full = api.wall_paged_attn(*args(table), window_size=50)
    gone = table.copy()
    gone[0, :(300 - 49) // 32] = -1
    gone[1, :(290 - 49) // 32] = -1
    assert torch.equal(full, api.wall_paged_attn(*args(gone), window_size=50))
    _status_ok()


def test_attn_shared_pages():
    """Two requests over the same prefix pages."""
    x, cu, kv, table = _attn_inputs(2, 1, 128, 128, 64, BF, [1, 1], [150, 150])
    t2 = table.copy()
    t2[1, :2] = t2[0, :2]
    o_ref, _ = ref.attn(x["q"], x["p"], cu, kv, torch.tensor(t2), x["k_pages"], x["v_pages"],
                        x["r_pages"], 64, 128 ** -0.5)
    o = api.wall_paged_attn(x["q"], x["p"], _i32(cu), _i32(kv), _i32(t2), x["k_pages"],
                            x["v_pages"], x["r_pages"], max_new=1)
    assert_fwd(BF, o, o_ref)


def test_attn_is_repeatable():
    x, cu, kv, table = _attn_inputs(4, 2, 128, 128, 64, BF, [1, 200, 3, 1], [2000, 900, 700, 64])
    call = lambda: api.wall_paged_attn(x["q"], x["p"], _i32(cu), _i32(kv), _i32(table),
                                       x["k_pages"], x["v_pages"], x["r_pages"], return_lse=True)
    first = call()
    for _ in range(3):
        for a, b in zip(first, call()):
            assert torch.equal(a, b)


# ----------------------------------------------------------- the steps in a row

@pytest.mark.parametrize("K,dt,PS,window", [(128, BF, 64, 0), (64, BF, 32, 100), (64, F32, 64, 0)])
def test_serving_run_matches_the_oracle(K, dt, PS, window):
    """Prompts in chunks, single tokens, drafts, a release and a new request in
    the freed row: every step's rows equal the oracle's forward of the whole
    sequence at those positions."""
    HQ, H = 4, 2
    gen = torch.Generator().manual_seed(11)
    lens = [230, 150, 170, 90]
    seqs = [dict(q=_rand(gen, n, HQ, K, dtype=dt), k=_rand(gen, n, H, K, dtype=dt),
                 v=_rand(gen, n, H, K, dtype=dt), g=-_rand(gen, n, HQ, K, dtype=dt, amp=0.04).abs())
            for n in lens]
    want = []
    for s in seqs:
        one = {n: t[None].cpu() for n, t in s.items()}
        want.append(wo.forward(one["q"], one["k"], one["v"], one["g"], scale=K ** -0.5,
                               window_size=window or None)[0][0])
    tb = api.WallPagedTables(3, 8, 24, page_size=PS)  # every row full at once
    cache = api.WallPagedCache(tb, H, HQ, K, K, dtype=dt, window_size=window or None)
    row_of, at = {0: 0, 1: 1, 2: 2}, [0] * 4
    steps = [[100, 1, 0], [1, 70, 130], [1, 1, 1], [60, 5, 1], [1, 73, 2], [1, 0, 36]]
    def step(new, seq_of):
        rows = [(i, seq_of[i], n) for i, n in enumerate(new) if n]
        cat = {x: torch.cat([seqs[s][x][at[s]:at[s] + n] for _, s, n in rows]) for x in "qkvg"}
        plan = tb.plan(_i32(new), sum(new))
        o = cache.step(plan, cat["q"], cat["k"], cat["v"], cat["g"], max_new=max(new))
        r0 = 0
        for i, s, n in rows:
            assert_fwd(dt, o[r0:r0 + n], want[s][at[s]:at[s] + n], what=f"request {i}")
            at[s] += n
            r0 += n
    for new in steps:
        step(new, row_of)
    tb.release(_i32([0, 1, 0]))       # request 1 is done; another takes its row
    row_of = {0: 0, 1: 3, 2: 2}
    for new in ([1, 60, 0], [0, 1, 0], [65, 29, 0]):
        step(new, row_of)
    assert at == [230, 150, 170, 90]
    _status_ok()


def test_captured_step_replays_with_new_lengths():
    """One CUDA graph of plan + append + attend serves every step of a fixed
    row count: the lengths, offsets and pages are read on the GPU."""
    HQ, H, K, PS, N, T = 4, 2, 128, 64, 3, 16
    gen = torch.Generator().manual_seed(21)
    new_steps = [[1, 9, 3], [4, 0, 1], [1, 1, 1], [7, 2, 7], [0, 0, 5]]
    x = [dict(q=_rand(gen, T, HQ, K), k=_rand(gen, T, H, K), v=_rand(gen, T, H, K),
              g=-_rand(gen, T, HQ, K, amp=0.04).abs()) for _ in new_steps]
    def fresh():
        tb = api.WallPagedTables(N, 4, 12, page_size=PS)
        return tb, api.WallPagedCache(tb, H, HQ, K, K)
    tb, cache = fresh()
    want = []
    for new, s in zip(new_steps, x):
        want.append(cache.step(tb.plan(_i32(new), T), s["q"], s["k"], s["v"], s["g"])[:sum(new)])
    tb, cache = fresh()
    buf = {n: t.clone() for n, t in x[0].items()}
    new_buf = _i32([0, 0, 0])
    run = lambda: cache.step(tb.plan(new_buf, T), buf["q"], buf["k"], buf["v"], buf["g"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for new, s, w in zip(new_steps, x, want):
        new_buf.copy_(_i32(new))
        for n in "qkvg":
            buf[n].copy_(s[n])
        graph.replay()
        assert torch.equal(out[:sum(new)], w)
    assert torch.equal(tb.lens, _i32([13, 12, 17]))
    _status_ok()


def test_two_streams_at_once():
    """Two caches stepped on two streams at the same time."""
    def make(seed):
        x, cu, kv, table = _attn_inputs(4, 2, 128, 128, 64, BF, [1, 64, 1], [900, 500, 300], seed)
        return lambda: api.wall_paged_attn(x["q"], x["p"], _i32(cu), _i32(kv), _i32(table),
                                           x["k_pages"], x["v_pages"], x["r_pages"])
    calls = [make(s) for s in (1, 2)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(5):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(c())
    torch.cuda.synchronize()
    for n, g in enumerate(got):
        assert torch.equal(g, want[n % 2])
    _status_ok()


def test_strided_inputs():
    """q, k, v, g as slices of one fused projection."""
    HQ, H, K, PS = 2, 1, 64, 32
    gen = torch.Generator().manual_seed(31)
    fused = _rand(gen, 50, 2 * HQ + 2 * H, K)
    q, g, k, v = fused[:, :HQ], -fused[:, HQ:2 * HQ].abs() * 0.02, fused[:, 2 * HQ:2 * HQ + H], fused[:, 2 * HQ + H:]
    outs = []
    for f in (lambda t: t, lambda t: t.contiguous()):
        tb = api.WallPagedTables(1, 2, 3, page_size=PS)
        c = api.WallPagedCache(tb, H, HQ, K, K)
        outs.append(c.step(tb.plan(_i32([50]), 50), f(q), f(k), f(v), f(g)))
    assert torch.equal(outs[0], outs[1])
