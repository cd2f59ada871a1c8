"""CPU tests of the paged cache: the header from C, the argument checks of the
library and of the Python API (the library takes bare pointers, so a wrong
shape or dtype must be refused before any call), and the division of a ragged
batch's tiles over a grid, restated on the host against counting."""
import os
import random
import re
import shutil
import subprocess

import pytest
import torch

from channel_decay_softmax_b200 import _lib as L
from channel_decay_softmax_b200 import api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "channel_decay_softmax_b200")
BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
HOST = "libwall takes CUDA tensors"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from channel_decay_softmax_b200 import build
    build.build()


def _declared():
    src = open(os.path.join(ROOT, "include", "wall_paged.h")).read()
    return sorted(set(re.findall(r"^\s*(?:int|size_t)\s+(wall_\w+)\s*\(", src, flags=re.M)))


def test_exports_every_declared_symbol():
    assert set(_declared()) == set(L.PAGED_EXPORTS)
    for n in _declared():
        assert hasattr(L.lib(), n), n


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_header_compiles_as_c_and_links(tmp_path):
    exe = tmp_path / "abi_check_paged"
    src = os.path.join(ROOT, "tests", "abi_check_paged.c")
    cc = ["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
          src, "-L", PKG, "-lwall", "-Wl,-rpath," + PKG, "-o", str(exe)]
    res = subprocess.run(cc, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr
    assert not [n for n in _declared() if f"(any_fn){n}" not in open(src).read()]
    assert f"ok ({len(_declared())} entry points)" in run.stdout


N, T, MP, NP, PS, H, HQ, K, V = 3, 7, 4, 9, 64, 2, 4, 64, 64


def _i(*shape):
    return torch.zeros(*shape, dtype=I32)


def _plan_args(**over):
    a = dict(new_lens=_i(N), lens=_i(N), block_table=_i(N, MP), free_list=_i(NP),
             free_count=_i(1), page_size=PS, n_tokens=T)
    a.update(over)
    return a


def _append_args(**over):
    a = dict(k=torch.zeros(T, H, K, dtype=BF), v=torch.zeros(T, H, V, dtype=BF),
             g=torch.zeros(T, HQ, K, dtype=BF), cu_q=_i(N + 1), kv_lens=_i(N),
             slot_map=torch.zeros(T, dtype=I64), k_pages=torch.zeros(NP, HQ, PS, K, dtype=BF),
             v_pages=torch.zeros(NP, H, PS, V, dtype=BF), r_pages=_i(NP, HQ, K),
             carry=torch.zeros(N, HQ, K, dtype=I64))
    a.update(over)
    return a


def _attn_args(**over):
    a = dict(q=torch.zeros(T, HQ, K, dtype=BF), p=torch.zeros(T, HQ, K), cu_q=_i(N + 1),
             kv_lens=_i(N), block_table=_i(N, MP), k_pages=torch.zeros(NP, HQ, PS, K, dtype=BF),
             v_pages=torch.zeros(NP, H, PS, V, dtype=BF), r_pages=_i(NP, HQ, K))
    a.update(over)
    return a


def test_well_formed_calls_pass_the_checks():
    for fn, args in ((api.wall_paged_plan, _plan_args()), (api.wall_paged_append, _append_args()),
                     (api.wall_paged_attn, _attn_args(sink_bias=torch.zeros(HQ), max_new=1)),
                     (api.wall_paged_release, dict(finished=_i(N), lens=_i(N),
                                                   block_table=_i(N, MP), free_list=_i(NP),
                                                   free_count=_i(1), page_size=PS))):
        with pytest.raises(ValueError, match=HOST):
            fn(**args)


@pytest.mark.parametrize("over", [
    dict(page_size=48), dict(page_size=16), dict(new_lens=_i(N + 1)),
    dict(new_lens=torch.zeros(N, dtype=I64)), dict(lens=_i(N, 1)), dict(block_table=_i(N * MP)),
    dict(free_list=torch.zeros(NP, dtype=I64)), dict(free_count=_i(2)), dict(n_tokens=-1),
    dict(lens_out=_i(N + 1)), dict(free_count_out=_i(2)), dict(block_table=_i(N, 0))])
def test_plan_refuses(over):
    with pytest.raises((TypeError, ValueError)) as e:
        api.wall_paged_plan(**_plan_args(**over))
    assert HOST not in str(e.value)


@pytest.mark.parametrize("over", [
    dict(k=torch.zeros(T, H, K)), dict(k=torch.zeros(1, T, H, K, dtype=BF)),
    dict(v=torch.zeros(T, H, V + 8, dtype=BF)), dict(g=torch.zeros(T, H, K, dtype=BF)),
    dict(g=torch.zeros(T, HQ, K, dtype=torch.float16)), dict(cu_q=_i(N)),
    dict(kv_lens=torch.zeros(N, dtype=I64)), dict(slot_map=_i(T)),
    dict(slot_map=torch.zeros(T + 1, dtype=I64)), dict(r_pages=torch.zeros(NP, HQ, K)),
    dict(k_pages=torch.zeros(NP, HQ, 48, K, dtype=BF)),
    dict(v_pages=torch.zeros(NP, 3, PS, V, dtype=BF)), dict(carry=torch.zeros(N, HQ, K)),
    dict(carry_out=torch.zeros(N, HQ, K)), dict(max_new=0)])
def test_append_refuses(over):
    with pytest.raises((TypeError, ValueError)) as e:
        api.wall_paged_append(**_append_args(**over))
    assert HOST not in str(e.value)


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(T, HQ, K)), dict(q=torch.zeros(T, HQ + 1, K, dtype=BF)),
    dict(p=torch.zeros(T, HQ, K, dtype=BF)), dict(p=torch.zeros(T - 1, HQ, K)),
    dict(cu_q=torch.zeros(N + 1, dtype=I64)), dict(kv_lens=_i(N, 1)),
    dict(block_table=_i(N + 1, MP)), dict(block_table=torch.zeros(N, MP, dtype=I64)),
    dict(block_table=_i(N, 0)), dict(sink_bias=torch.zeros(HQ + 1)), dict(max_new=-3),
    dict(r_pages=_i(NP, H, K))])
def test_attn_refuses(over):
    with pytest.raises((TypeError, ValueError)) as e:
        api.wall_paged_attn(**_attn_args(**over))
    assert HOST not in str(e.value)


def test_tables_and_cache_refuse_bad_sizes():
    with pytest.raises(ValueError):
        api.WallPagedTables(0, 4, 4, device="cpu")
    with pytest.raises(ValueError):
        api.WallPagedTables(2, 4, 4, page_size=100, device="cpu")
    tb = api.WallPagedTables(2, 4, 6, page_size=32, device="cpu")
    assert tb.free_list.tolist() == [5, 4, 3, 2, 1, 0] and tb.free_count.item() == 6
    with pytest.raises(ValueError):
        api.WallPagedCache(tb, H=2, HQ=3, K=64, V=64)


FAKE = 4096


def test_library_refuses_bad_arguments():
    lib = L.lib()
    ap = lambda HQ=4, K=64, dtype=0, ps=64, k=FAKE, carry=FAKE, mx=0: lib.wall_paged_append(
        k, FAKE, FAKE, dtype, FAKE, FAKE, FAKE, 2, 5, mx, 2, HQ, K, 64, ps, 8, FAKE, FAKE, FAKE,
        carry, FAKE, FAKE, None, 0, None)
    assert ap(HQ=3) == L.WALL_ERR_INVALID_ARG
    assert ap(dtype=2) == L.WALL_ERR_INVALID_ARG
    assert ap(mx=-1) == L.WALL_ERR_INVALID_ARG
    assert ap(K=100) == L.WALL_ERR_UNSUPPORTED
    assert ap(K=256) == L.WALL_ERR_UNSUPPORTED
    assert ap(ps=16) == L.WALL_ERR_UNSUPPORTED
    assert ap(HQ=8192) == L.WALL_ERR_UNSUPPORTED
    assert ap(k=None) == L.WALL_ERR_INVALID_ARG
    assert ap(k=FAKE + 8) == L.WALL_ERR_INVALID_ARG
    assert ap(carry=FAKE + 8) == L.WALL_ERR_INVALID_ARG
    need = lib.wall_paged_attn_workspace(0, 2, 5, 0, 2, 4, 64, 64)
    assert need > 0 and lib.wall_paged_attn_workspace(0, 2, 5, 0, 2, 3, 64, 64) == 0
    at = lambda q=FAKE, table=FAKE, mp=4, ws=FAKE, nb=need, V=64, NPg=8: lib.wall_paged_attn(
        q, FAKE, 0, FAKE, FAKE, table, 2, 5, 0, mp, 2, 4, 64, V, 64, NPg, FAKE, FAKE, FAKE, None,
        0.0, 0, FAKE, None, ws, nb, None)
    assert at(q=None) == L.WALL_ERR_INVALID_ARG
    assert at(table=None) == L.WALL_ERR_INVALID_ARG
    assert at(table=FAKE + 2) == L.WALL_ERR_INVALID_ARG
    assert at(mp=0) == L.WALL_ERR_INVALID_ARG
    assert at(ws=None) == L.WALL_ERR_INVALID_ARG
    assert at(nb=need - 1) == L.WALL_ERR_INVALID_ARG
    assert at(V=132) == L.WALL_ERR_UNSUPPORTED
    assert at(NPg=0) == L.WALL_ERR_INVALID_ARG
    assert at(NPg=1 << 24) == L.WALL_ERR_UNSUPPORTED


# ---- the division of the tiles (wall_paged.cuh), restated

class Req:
    def __init__(self, n, kv, window, TB):
        self.n, self.ctx, self.dead, self.TB = n, kv - n, kv < n, TB
        self.nb = -(-n // TB)
        self.c1 = (self.ctx + TB - 1) // TB
        self.last = (self.ctx + n - 1) // TB
        self.f = (self.ctx - window + 1) // TB if window else -(1 << 28)

    def lo(self, b):
        return 0 if self.dead else max(0, b + self.f)

    def hi(self, b):
        return 0 if self.dead else (b + self.c1 if b < self.nb - 1 else self.last)

    def tiles(self, b):
        return self.hi(b) - self.lo(b) + 1

    def before(self, m):
        if self.dead:
            return m
        s = m * (m - 1) // 2 + m * (self.c1 + 1)
        k = m - 1 + self.f
        if k > 0:
            lo = self.f if self.f > 0 else 1
            s -= (lo + k) * (k - lo + 1) // 2
        return s


@pytest.mark.parametrize("TB", [32, 128])
def test_unit_tiles_are_the_visible_ones(TB):
    rng = random.Random(5)
    for _ in range(400):
        n = rng.choice([1, 2, 31, 32, 33, 127, 128, 129, 300, rng.randint(1, 900)])
        ctx = rng.choice([0, 1, 31, 32, 127, 128, 129, rng.randint(0, 2000)])
        w = rng.choice([0, 1, 2, 31, 33, 128, 129, rng.randint(1, 1500)])
        r = Req(n, ctx + n, w, TB)
        total = 0
        for b in range(r.nb):
            assert r.before(b) == total
            i0, i1 = ctx + b * TB, ctx + min(n, (b + 1) * TB) - 1
            first = max(0, i0 - w + 1) if w else 0
            assert (r.lo(b), r.hi(b)) == (first // TB, i1 // TB), (n, ctx, w, b)
            total += r.tiles(b)


@pytest.mark.parametrize("U", [0, 1, 3])
def test_every_tile_has_one_owner(U):
    """Units of U + tiles places each, cut into even shares: every tile falls to
    the one CTA that holds its place, a unit's tiles to neighbours, and the CTA
    that ends a unit is the one its beginner names."""
    rng = random.Random(6)
    for _ in range(150):
        units = [rng.randint(1, 40) for _ in range(rng.randint(1, 60))]
        W = sum(U + n for n in units)
        G = min(W, rng.randint(1, 300))
        begin = [W * c // G for c in range(G + 1)]
        owner = lambda x: ((x + 1) * G + W - 1) // W - 1
        for c in range(G):
            assert all(owner(x) == c for x in range(begin[c], begin[c + 1]))
        got = [[] for _ in units]  # (CTA, ta, tb) of each unit
        for c in range(G):
            x, base = begin[c], 0
            for u, n in enumerate(units):
                if base + U + n > begin[c] and base < begin[c + 1]:
                    p = max(begin[c], base) - base
                    places = min(begin[c + 1] - base - p, U + n - p)
                    ta, tb = max(0, p - U), max(0, p + places - U)
                    if tb > ta:
                        got[u].append((c, ta, tb, owner(base + U + n - 1)))
                base += U + n
        for n, runs in zip(units, got):
            assert runs[0][1] == 0 and runs[-1][2] == n
            assert all(a[2] == b[1] and a[0] + 1 == b[0] for a, b in zip(runs, runs[1:]))
            assert runs[0][3] == runs[-1][0]
