"""Cases of the paged-cache operators: the page plan of a serving step, the
append of its tokens to the paged Wall cache, the attention of the new tokens
over the pages, and the three in a row as a serving loop runs them.

Shapes shared by all cases
  N requests, request i with ctx_i cached tokens and q_i new ones, packed back
  to back: q, g [T, HQ, K], k [T, H, K], v [T, H, V], cu_q [N + 1] int32.
  Pools of pages of PS positions: k_pages [NP, HQ, PS, K], v_pages
  [NP, H, PS, V], r_pages [NP, HQ, K] int32 (each page's integer anchors);
  block_table [N, MP] int32 gives request i's pages in order (-1: none).

The decay's prefix is held in fixed point, 24 fraction bits, in powers of two:
  e_t = rint(g_t * 2^24 / ln 2) (fp32 product, clamped to 32 signed bits),
  P_t = P_{t-1} + e_t (64-bit integers, exact in every order),
  R_c = floor(P / 2^24 + 1/2) at page c's first position,
  p_t = P_t / 2^24 - R_{page(t)}            (what append returns, fp32)
  k_pages row of t = k_t * 2^(-p_t)
  s_ij = scale * sum_n q_in 2^(p_in + R_{page(i),n} - R_{page(j),n}) k_pages_jn
"""
import math
import random

import torch

own = False

DEV = "cuda"
FRAC = 24
ONE = 1 << FRAC
C_FIX = 16777216.0 / math.log(2.0)
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # a serving loop's bookkeeping: a handful of requests, one token each
        # but for a prompt that arrives
        dict(name="plan 5 requests", op="plan", N=5, new_lo=1, new_hi=33, ctx_lo=0, ctx_hi=500,
             PS=32, lens=1),
        # a large batch with prompts among it, 2048 rows of the block table
        dict(name="plan 2048 requests", op="plan", N=2048, new_lo=1, new_hi=60, ctx_lo=0,
             ctx_hi=9000, PS=64, lens=2),
        # one decode step's tokens of 48 requests (heads as the decode workload)
        dict(name="append decode 48", op="append", N=48, new_lo=1, new_hi=1, ctx_lo=1,
             ctx_hi=4000, HQ=32, H=8, K=128, V=128, PS=64, type="bf16", lens=3),
        # prompts of several requests at once, ragged (heads of the T = 8192 workload)
        dict(name="append prompts bf16", op="append", N=6, new_lo=301, new_hi=2500, ctx_lo=0,
             ctx_hi=700, HQ=16, H=4, K=128, V=128, PS=64, type="bf16", lens=4),
        # the fp32 form, odd head counts, lengths around a page
        dict(name="append fp32", op="append", N=9, new_lo=1, new_hi=150, ctx_lo=0, ctx_hi=130,
             HQ=6, H=3, K=64, V=64, PS=32, type="fp32", lens=5),
        # the smallest decode: three short conversations
        dict(name="attn decode 3", op="attn", N=3, new_lo=1, new_hi=1, ctx_lo=10, ctx_hi=300,
             HQ=8, H=4, K=64, V=64, PS=32, type="bf16", window=0, sink=True, lens=6),
        # a decode batch with long ragged contexts (heads of the decode workload)
        dict(name="attn decode 32 long", op="attn", N=32, new_lo=1, new_hi=1, ctx_lo=4096,
             ctx_hi=16000, HQ=32, H=8, K=128, V=128, PS=64, type="bf16", window=0, sink=False,
             lens=7),
        # several tokens a request: drafts to be verified
        dict(name="attn drafts 16", op="attn", N=16, new_lo=2, new_hi=8, ctx_lo=1900,
             ctx_hi=9000, HQ=16, H=4, K=128, V=128, PS=128, type="bf16", window=0, sink=False,
             lens=8),
        # chunks of prompts over what is cached, with the window and the sink of
        # the packed workload
        dict(name="attn chunks window", op="attn", N=5, new_lo=200, new_hi=1001, ctx_lo=500,
             ctx_hi=4000, HQ=16, H=2, K=128, V=128, PS=64, type="bf16", window=1024, sink=True,
             lens=9),
        # one whole prompt of 8192 tokens
        dict(name="attn prompt 8192", op="attn", N=1, new_lo=8192, new_hi=8192, ctx_lo=0,
             ctx_hi=0, HQ=16, H=4, K=128, V=128, PS=64, type="bf16", window=0, sink=False,
             lens=10),
        # fp32, a small model's chunk beside single tokens
        dict(name="attn fp32", op="attn", N=6, new_lo=1, new_hi=70, ctx_lo=0, ctx_hi=900, HQ=4,
             H=2, K=64, V=64, PS=32, type="fp32", window=0, sink=True, lens=11),
        # a serving step as it is run: mostly single tokens, two chunks of prompts
        dict(name="step mixed", op="step", N=24, new_lo=1, new_hi=1, n_long=2, long_lo=200,
             long_hi=700, ctx_lo=30, ctx_hi=3000, HQ=16, H=4, K=128, V=128, PS=64, type="bf16",
             window=0, sink=False, lens=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attn", "attn", "attn", "step"])
    PS = rng.choice([32, 64, 128])
    lens = rng.randrange(100, 1 << 30)
    if op == "plan":
        hi = _log_int(rng, 1, 60)
        return dict(op=op, N=_log_int(rng, 1, 2000), new_lo=rng.choice([0, 1]), new_hi=hi,
                    ctx_lo=0, ctx_hi=_log_int(rng, 10, 9000), PS=PS, lens=lens)
    kind = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    H = rng.choice([1, 2, 3, 4])
    G = rng.choice([1, 2, 4])
    D = rng.choice([64, 128])
    K, V = (D, D) if rng.random() < 0.8 else (rng.choice([64, 128]), rng.choice([64, 128]))
    base = dict(op=op, HQ=H * G, H=H, K=K, V=V, PS=PS, type=kind, lens=lens)
    decode = rng.random() < 0.4
    if op == "append":
        N = _log_int(rng, 1, 200) if decode else _log_int(rng, 1, 10)
        hi = 1 if decode else _log_int(rng, 2, 1500)
        return dict(base, N=N, new_lo=1, new_hi=hi, ctx_lo=0, ctx_hi=_log_int(rng, 20, 2000))
    if op == "step":
        return dict(base, N=_log_int(rng, 2, 24), new_lo=1, new_hi=1, n_long=rng.choice([0, 1, 2]),
                    long_lo=2, long_hi=_log_int(rng, 10, 600), ctx_lo=0,
                    ctx_hi=_log_int(rng, 50, 2500), window=rng.choice([0, 0, 300]),
                    sink=rng.random() < 0.5)
    if kind == "fp32":
        N, hi, ctx = _log_int(rng, 1, 8), 1 if decode else _log_int(rng, 2, 100), _log_int(rng, 20, 900)
    elif decode:
        N, hi, ctx = _log_int(rng, 1, 32), 1, _log_int(rng, 50, 9000)
    else:
        N, hi, ctx = _log_int(rng, 1, 6), _log_int(rng, 2, 900), _log_int(rng, 20, 3500)
    return dict(base, N=N, new_lo=1, new_hi=hi, ctx_lo=0, ctx_hi=ctx,
                window=rng.choice([0, 0, 200, 1024]), sink=rng.random() < 0.5)


def _lengths(case):
    """(ctx, new) of every request: the case's own numbers, whatever the seed."""
    rng = random.Random(case["lens"])
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["N"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["N"])]
    for i in range(case.get("n_long", 0)):
        new[(i * 7 + 3) % case["N"]] = rng.randint(case["long_lo"], case["long_hi"])
    if sum(new) == 0:
        new[0] = 1
    return ctx, new


# -------------------------------------------------------------------- inputs

def _table(ctx, new, PS, gen, spare=3):
    """Block table whose held pages are a random choice of the pool, and the
    stack of the free ones: (table, free_list, free_count, pages needed at most)."""
    N = len(ctx)
    held = [-(-c // PS) for c in ctx]
    want = [-(-(c + n) // PS) for c, n in zip(ctx, new)]
    MP = max(1, max(want))
    NP = sum(want) + spare
    perm = torch.randperm(NP, generator=gen).to(torch.int32)
    held_t = torch.tensor(held)
    at = torch.cumsum(held_t, 0) - held_t
    j = torch.arange(MP)[None, :]
    inside = j < held_t[:, None]
    idx = torch.where(inside, at[:, None] + j, torch.zeros((), dtype=torch.long))
    table = torch.where(inside, perm[idx].long(), torch.full((), -1)).to(torch.int32)
    nheld = int(held_t.sum())
    free = torch.full((NP,), -1, dtype=torch.int32)
    free[:NP - nheld] = perm[nheld:]
    return table, free, NP - nheld, NP, MP


def _noise(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _gates(gen, shape, dtype):
    """g = -0.02 |N|, as the decode workload's gates."""
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).abs_() * -0.02).to(dtype)


def _pools(case, NP, table, gen):
    """Pools as they stand after the cached tokens of gates of 0.02 |N| were
    appended: anchors falling from page to page of a request, and key rows that
    grow by the decay inside a page (0.023 powers of two a token)."""
    HQ, H, K, V, PS = case["HQ"], case["H"], case["K"], case["V"], case["PS"]
    dt = TYPES[case["type"]]
    per_page = 0.023 * PS
    k_pages = torch.empty((NP, HQ, PS, K), dtype=dt, device=DEV)
    grow = torch.exp2(0.023 * torch.arange(PS, device=DEV, dtype=torch.float32))[:, None]
    step = max(1, (1 << 27) // (HQ * PS * K))
    for a in range(0, NP, step):
        b = min(NP, a + step)
        k_pages[a:b] = _noise(gen, (b - a, HQ, PS, K), torch.float32) * grow
    v_pages = _noise(gen, (NP, H, PS, V), dt)
    r_pages = torch.zeros((NP, HQ, K), dtype=torch.int32, device=DEV)
    t = table.to(DEV).long()
    ids, at = t[t >= 0], torch.arange(t.shape[1], device=DEV).expand_as(t)[t >= 0]
    tilt = 0.7 + 0.6 * torch.rand((HQ, K), generator=gen, device=DEV)
    r_pages[ids] = torch.floor(-per_page * at[:, None, None] * tilt + 0.5).to(torch.int32)
    return k_pages, v_pages, r_pages, tilt


def prepare(case, seed):
    host = torch.Generator().manual_seed(int(seed))
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    ctx, new = _lengths(case)
    N, PS, T = case["N"], case["PS"], sum(new)
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(new), 0)
    st = dict(case=case, N=N, PS=PS, T=T, max_new=max(new), op=case["op"])
    with_plan = case["op"] in ("plan", "step")
    # before a plan the table holds the cached tokens' pages; behind it, all
    table, free, n_free, NP, MP = _table(ctx if with_plan else [c + n for c, n in zip(ctx, new)],
                                         new if with_plan else [0] * N, PS, host)
    st.update(table=table.to(DEV), NP=NP, MP=MP)
    if with_plan:
        st.update(new_lens=torch.tensor(new, dtype=torch.int32).to(DEV),
                  lens=torch.tensor(ctx, dtype=torch.int32).to(DEV), free_list=free.to(DEV),
                  free_count=torch.tensor([n_free], dtype=torch.int32).to(DEV),
                  lens_out=torch.zeros(N, dtype=torch.int32, device=DEV),
                  free_out=torch.zeros(1, dtype=torch.int32, device=DEV))
    if case["op"] == "plan":
        return st
    HQ, H, K, V = case["HQ"], case["H"], case["K"], case["V"]
    dt = TYPES[case["type"]]
    st["k_pages"], st["v_pages"], st["r_pages"], tilt = _pools(case, NP, table, gen)
    kv = torch.tensor([c + n for c, n in zip(ctx, new)], dtype=torch.int32).to(DEV)
    if case["op"] != "step":
        st.update(cu_q=cu.to(DEV), kv_lens=kv)
    if case["op"] in ("append", "step"):
        st.update(k=_noise(gen, (T, H, K), dt), v=_noise(gen, (T, H, V), dt),
                  g=_gates(gen, (T, HQ, K), dt))
        # the prefix at the last cached token: inside its page's decay
        c = torch.tensor(ctx, device=DEV)
        last = (c - 1).clamp(min=0)
        page = st["table"][torch.arange(N, device=DEV), last // PS].clamp(min=0).long()
        off = (last % PS).to(torch.float64)[:, None, None] * 0.023 * tilt.double()
        carry = (st["r_pages"][page].to(torch.int64) << FRAC) - torch.floor(off * ONE).to(torch.int64)
        st["carry"] = torch.where((c > 0)[:, None, None], carry, torch.zeros_like(carry))
        st["carry_out"] = torch.zeros_like(st["carry"])
    if case["op"] == "append":
        st["slot_map"] = _slots(st["table"], st["cu_q"], kv, T, PS)
    if case["op"] in ("attn", "step"):
        st["q"] = _noise(gen, (T, HQ, K), dt)
        st["sink"] = _noise(gen, (HQ,), torch.float32) if case["sink"] else None
        st["window"] = case["window"]
        st["scale"] = K ** -0.5
    if case["op"] == "attn":
        pos = _positions(st["cu_q"], kv, T)[1]
        st["p"] = ((pos % PS).float()[:, None, None] * (-0.023 * tilt)
                   - 0.4 * torch.rand((T, HQ, K), generator=gen, device=DEV))
    return st


# --------------------------------------------------------------- plain forms

def _positions(cu_q, kv_lens, T):
    """(request, position) of every packed token."""
    t = torch.arange(T, device=cu_q.device)
    req = torch.searchsorted(cu_q[1:].long().contiguous(), t, right=True)
    ctx = kv_lens - (cu_q[1:] - cu_q[:-1])
    return req, ctx[req].long() + t - cu_q[req].long()


def _slots(table, cu_q, kv_lens, T, PS):
    req, pos = _positions(cu_q, kv_lens, T)
    return table[req, pos // PS].long() * PS + pos % PS


def _plain_plan(st):
    lens, new, table, PS, T = st["lens"].long(), st["new_lens"].long(), st["table"], st["PS"], st["T"]
    MP = table.shape[1]
    new = new.clamp(min=0)
    cu = torch.zeros(new.numel() + 1, dtype=torch.long, device=new.device)
    cu[1:] = torch.cumsum(new, 0)
    held, want = (lens + PS - 1) // PS, (lens + new + PS - 1) // PS
    fits = (want <= MP) & (cu[1:] <= T)
    need = torch.where(fits, want - held, torch.zeros_like(want))
    upto = torch.cumsum(need, 0)
    admitted = fits & ((need == 0) | (upto <= st["free_count"].long()))
    after = torch.where(admitted, lens + new, lens)
    used = torch.where(admitted, upto, torch.zeros_like(upto)).max()
    j = torch.arange(MP, device=new.device)[None, :]
    fresh = admitted[:, None] & (j >= held[:, None]) & (j < want[:, None])
    rank = (upto - need)[:, None] + j - held[:, None]
    pick = (st["free_count"].long() - 1 - rank).clamp(0, st["free_list"].numel() - 1)
    table.copy_(torch.where(fresh, st["free_list"][pick], table))
    st["lens_out"].copy_(after)
    st["free_out"].copy_(st["free_count"] - used)
    t = torch.arange(T, device=new.device)
    req = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=new.numel() - 1)
    pos = lens[req] + t - cu[req]
    page = table[req, (pos // PS).clamp(0, MP - 1)].long()
    slot = torch.where((t < cu[-1]) & admitted[req], page * PS + pos % PS, torch.full_like(pos, -1))
    return dict(cu_q=cu.to(torch.int32), slot_map=slot, admitted=admitted.to(torch.int32),
                kv_lens=torch.where(admitted, after, torch.zeros_like(after)).to(torch.int32))


def _plain_append(st, cu_q, kv_lens, slot_map):
    k, v, g, PS = st["k"], st["v"], st["g"], st["PS"]
    T, HQ, K = g.shape
    G = HQ // k.shape[1]
    req, pos = _positions(cu_q, kv_lens, T)
    first = cu_q[req].long()
    fixed = torch.tensor(C_FIX, dtype=torch.float32, device=g.device)
    e = torch.round(g.float() * fixed).double().clamp(-2147483648.0, 2147483647.0).to(torch.int64)
    run = torch.cumsum(e, 0)
    begun = (pos == torch.arange(T, device=g.device) - first)[:, None, None]  # nothing cached before
    before = torch.where(begun, torch.zeros_like(run[:1]), st["carry"][req])
    P = run - (run - e)[first] + before
    page, off = slot_map // PS, slot_map % PS
    opens = pos - off  # the page's first position, and its token where it is a new one
    token = torch.arange(T, device=g.device) - off
    inside = token >= first
    R = (P[token.clamp(min=0)] + (ONE >> 1)) >> FRAC
    R = torch.where(inside[:, None, None], R, st["r_pages"][page].long())
    p = (P - (R << FRAC)).float() * (1.0 / ONE)
    kt = k.float().repeat_interleave(G, dim=1) * torch.exp2(-p)
    st["k_pages"][page, :, off] = kt.to(k.dtype)
    st["v_pages"][page, :, off] = v
    st["r_pages"][page] = R.to(torch.int32)
    st["carry_out"].copy_(P[cu_q[1:].long() - 1])
    return p


def _plain_attn(st, p, cu_q, kv_lens):
    q, k_pages, v_pages, r_pages, table, PS = (st["q"], st["k_pages"], st["v_pages"], st["r_pages"],
                                               st["table"], st["PS"])
    T, HQ, K = q.shape
    NP, H, _, V = v_pages.shape
    N, MP, G, MQ = st["N"], table.shape[1], HQ // H, st["max_new"]
    dev = q.device
    qlen = cu_q[1:] - cu_q[:-1]
    m = torch.arange(MQ, device=dev)[None, :]
    rows = (cu_q[:-1, None] + m).clamp(max=T - 1).long()
    real = m < qlen[:, None]
    pos = (kv_lens - qlen)[:, None].long() + m
    bt = table.clamp(min=0).long()
    Rk = r_pages[bt]                                                       # [N, MP, HQ, K]
    here = (pos // PS).clamp(0, MP - 1)
    Rq = r_pages[bt.gather(1, here)]                                       # [N, MQ, HQ, K]
    ex = p[rows][:, :, None] + (Rq[:, :, None] - Rk[:, None]).float()      # [N, MQ, MP, HQ, K]
    old = torch.arange(MP, device=dev)[None, None, :] <= here[:, :, None]
    ex = torch.where(old[..., None, None], ex, torch.full((), -math.inf, device=dev))
    qs = torch.exp2(ex) * q.float()[rows][:, :, None]
    del ex
    s = torch.einsum("nmphk,nphjk->nhmpj", qs, k_pages[bt].float()).reshape(N, HQ, MQ, MP * PS)
    del qs
    j = torch.arange(MP * PS, device=dev)[None, None, :]
    seen = (j <= pos[:, :, None]) & (j < kv_lens[:, None, None])
    if st["window"] > 0:
        seen = seen & (j > pos[:, :, None] - st["window"])
    s = torch.where(seen[:, None], s * st["scale"], torch.full((), -math.inf, device=dev))
    top = s.amax(-1, keepdim=True)
    if st["sink"] is not None:
        top = torch.maximum(top, st["sink"].float()[None, :, None, None])
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    w = torch.exp(s - top)
    total = w.sum(-1, keepdim=True)
    if st["sink"] is not None:
        total = total + torch.exp(st["sink"].float()[None, :, None, None] - top)
    vv = v_pages[bt].float().permute(0, 2, 1, 3, 4).reshape(N, H, MP * PS, V)
    vv = torch.where(((j[0] < kv_lens[:, None])[:, None, :, None]), vv, torch.zeros((), device=dev))
    o = torch.einsum("nhgmj,nhjv->nhgmv", w.reshape(N, H, G, MQ, MP * PS), vv).reshape(N, HQ, MQ, V)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    return o.permute(0, 2, 1, 3)[real].to(q.dtype)


# ---------------------------------------------------------------------- runs

def _plan_of(st):
    if own:
        from channel_decay_softmax_b200 import wall_paged_plan
        pl = wall_paged_plan(st["new_lens"], st["lens"], st["table"], st["free_list"],
                             st["free_count"], page_size=st["PS"], n_tokens=st["T"],
                             lens_out=st["lens_out"], free_count_out=st["free_out"])
        return dict(cu_q=pl.cu_q, kv_lens=pl.kv_lens, slot_map=pl.slot_map, admitted=pl.admitted)
    return _plain_plan(st)


def _append_of(st, cu_q, kv_lens, slot_map):
    if own:
        from channel_decay_softmax_b200 import wall_paged_append
        return wall_paged_append(st["k"], st["v"], st["g"], cu_q, kv_lens, slot_map,
                                 st["k_pages"], st["v_pages"], st["r_pages"], st["carry"],
                                 carry_out=st["carry_out"], max_new=st["max_new"])
    return _plain_append(st, cu_q, kv_lens, slot_map)


def _attn_of(st, p, cu_q, kv_lens):
    if own:
        from channel_decay_softmax_b200 import wall_paged_attn
        return wall_paged_attn(st["q"], p, cu_q, kv_lens, st["table"], st["k_pages"],
                               st["v_pages"], st["r_pages"], max_new=st["max_new"],
                               scale=st["scale"], sink_bias=st["sink"],
                               window_size=st["window"])
    return _plain_attn(st, p, cu_q, kv_lens)


def run(st):
    if st["op"] == "plan":
        pl = _plan_of(st)
        return dict(pl, table=st["table"], lens=st["lens_out"], free_count=st["free_out"])
    if st["op"] == "append":
        p = _append_of(st, st["cu_q"], st["kv_lens"], st["slot_map"])
        return dict(p=p, k_pages=st["k_pages"], v_pages=st["v_pages"], r_pages=st["r_pages"],
                    carry=st["carry_out"])
    if st["op"] == "attn":
        return _attn_of(st, st["p"], st["cu_q"], st["kv_lens"])
    pl = _plan_of(st)
    p = _append_of(st, pl["cu_q"], pl["kv_lens"], pl["slot_map"])
    o = _attn_of(st, p, pl["cu_q"], pl["kv_lens"])
    return dict(o=o, p=p, k_pages=st["k_pages"], r_pages=st["r_pages"], carry=st["carry_out"],
                slot_map=pl["slot_map"], kv_lens=pl["kv_lens"], table=st["table"],
                lens=st["lens_out"], free_count=st["free_out"])


# ----------------------------------------------------------------- accounting

def _append_work(case, ctx, new):
    es = 2 if case["type"] == "bf16" else 4
    HQ, H, K, V, T = case["HQ"], case["H"], case["K"], case["V"], sum(new)
    opened = sum(-(-(c + n) // case["PS"]) - -(-c // case["PS"]) for c, n in zip(ctx, new))
    partly = sum(1 for c in ctx if c % case["PS"])
    b = T * (HQ * K * es + H * (K + V) * es)         # g, k, v read
    b += T * (HQ * K * (4 + es) + H * V * es)        # p, key and value rows written
    b += case["N"] * HQ * K * 16 + (opened + partly) * HQ * K * 4 + T * 8  # carries, anchors, slots
    return b, T * HQ * K * 6


def _attn_work(case, ctx, new):
    es = 2 if case["type"] == "bf16" else 4
    HQ, H, K, V, PS, W = case["HQ"], case["H"], case["K"], case["V"], case["PS"], case["window"]
    keys = pages = pairs = 0
    for c, n in zip(ctx, new):
        lo = max(0, c - W + 1) if W else 0
        keys += c + n - lo
        pages += -(-(c + n) // PS) - lo // PS
        if W:
            pairs += sum(min(c + i + 1, W) for i in range(n))
        else:
            pairs += n * c + n * (n + 1) // 2
    T = sum(new)
    b = keys * (HQ * K + H * V) * es + pages * HQ * K * 4 + T * HQ * (K * (4 + es) + V * es)
    return b, 2 * pairs * HQ * (K + V)


def work(case):
    ctx, new = _lengths(case)
    N, T, PS = case["N"], sum(new), case["PS"]
    opened = sum(-(-(c + n) // PS) - -(-c // PS) for c, n in zip(ctx, new))
    b = f = 0
    if case["op"] in ("plan", "step"):
        b, f = b + 28 * N + 8 * T + 8 * opened, f + 8 * N + 4 * T
    if case["op"] in ("append", "step"):
        x = _append_work(case, ctx, new)
        b, f = b + x[0], f + x[1]
    if case["op"] in ("attn", "step"):
        x = _attn_work(case, ctx, new)
        b, f = b + x[0], f + x[1]
    return dict(bytes=b, flops=f)


# -------------------------------------------------------------------- 64 bits

def _exact_append(st, ctx, new, table):
    """p, key pages and value pages in 64 bits, request by request."""
    PS, G = st["PS"], st["case"]["HQ"] // st["case"]["H"]
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    rp = st["r_pages"].double()
    ps, t0 = [], 0
    c32 = torch.tensor(C_FIX, dtype=torch.float32, device=DEV)
    for i, (c, n) in enumerate(zip(ctx, new)):
        if n == 0:
            continue
        e = torch.round(st["g"][t0:t0 + n].float() * c32).double().clamp(-2.0 ** 31, 2.0 ** 31 - 1)
        start = st["carry"][i].double() if c > 0 else torch.zeros_like(st["carry"][i]).double()
        P = (torch.cumsum(e, 0) + start) / ONE     # sums of integers below 2^53: exact
        at = torch.arange(c, c + n, device=DEV)
        page = table[i][at // PS].long()
        for d in range(c // PS, (c + n - 1) // PS + 1):
            if d * PS >= c:
                rp[table[i][d].long()] = torch.floor(P[d * PS - c] + 0.5)
        p = P - rp[page]
        kp[page, :, at % PS] = st["k"][t0:t0 + n].double().repeat_interleave(G, 1) * torch.exp2(-p)
        vp[page, :, at % PS] = st["v"][t0:t0 + n].double()
        ps.append(p)
        t0 += n
    return torch.cat(ps), kp, vp, rp


def _exact_attn(st, p, kp, vp, rp, ctx, new, table):
    case, PS = st["case"], st["PS"]
    G = case["HQ"] // case["H"]
    outs, t0 = [], 0
    for i, (c, n) in enumerate(zip(ctx, new)):
        if n == 0:
            continue
        L = c + n
        ids = table[i][:-(-L // PS)].long()
        vv = vp[ids].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :L]
        o = torch.empty((n, case["HQ"], case["V"]), dtype=torch.float64, device=DEV)
        at = torch.arange(c, L, device=DEV)
        j = torch.arange(L, device=DEV)
        seen = j[None, :] <= at[:, None]
        if st["window"] > 0:
            seen &= at[:, None] - j[None, :] < st["window"]
        far = p[t0:t0 + n].double() + rp[ids[at // PS]].double()
        for h in range(case["HQ"]):
            s = torch.full((n, ids.numel() * PS), -math.inf, dtype=torch.float64, device=DEV)
            x = st["q"][t0:t0 + n, h].double()
            if n <= 64:                            # all pages at once
                y = x * torch.exp2(far[:, h] - rp[ids, None, h].double())
                s = torch.bmm(y, kp[ids, h].double().mT).permute(1, 0, 2).reshape(n, -1)
            else:
                for d in range(ids.numel()):
                    r0 = max(0, d * PS - c)        # rows that can see the page
                    y = x[r0:] * torch.exp2(far[r0:, h] - rp[ids[d], h].double())
                    s[r0:, d * PS:(d + 1) * PS] = y @ kp[ids[d], h].double().T
            s = (s[:, :L] * case["K"] ** -0.5).masked_fill(~seen, -math.inf)
            if st["sink"] is not None:
                s = torch.cat([s, st["sink"][h].double().expand(n, 1)], 1)
            o[:, h] = torch.softmax(s, 1)[:, :L] @ vv[h // G]
        outs.append(o)
        t0 += n
    return torch.cat(outs)


def exact(case, seed):
    if case["op"] == "plan":
        return None
    ctx, new = _lengths(case)
    PS = case["PS"]
    st = prepare(case, seed)
    table = st["table"]
    if case["op"] == "attn":
        return _exact_attn(st, st["p"], st["k_pages"], st["v_pages"], st["r_pages"], ctx, new, table)
    if case["op"] == "step":
        table = table.clone()                      # pages from the stack's end, request by request
        n_free = int(st["free_count"][0])
        for i, (c, n) in enumerate(zip(ctx, new)):
            for d in range(-(-c // PS), -(-(c + n) // PS)):
                n_free -= 1
                table[i, d] = st["free_list"][n_free]
    p, kp, vp, rp = _exact_append(st, ctx, new, table)
    if case["op"] == "append":
        return dict(p=p, k_pages=kp, v_pages=vp, r_pages=None, carry=None)
    # the attention reads the key rows as the cache holds them
    held = kp.to(TYPES[case["type"]])
    o = _exact_attn(st, p, held, vp, rp, ctx, new, table)
    return dict(o=o, p=p, k_pages=kp, r_pages=None, carry=None, slot_map=None, kv_lens=None,
                table=None, lens=None, free_count=None)
