"""The paged-cache operators in 64 bits, request by request, for the tests.
Shares no code with the CUDA path: the decay is applied as the running product
of the gates in float64, with the fixed-point gate of the definition."""
import math

import numpy as np
import torch

FRAC = 24
C32 = np.float32(np.float32(1.4426950408889634) * np.float32(1 << FRAC))


def f64(t):
    return t.detach().float().cpu().double().numpy() if t.dtype == torch.bfloat16 \
        else t.detach().cpu().double().numpy()


def gate_steps(g):
    """e_t of gates g, int64."""
    x = np.rint(g.detach().float().cpu().numpy() * C32).astype(np.float64)
    return np.clip(x, -2.0 ** 31, 2.0 ** 31 - 1).astype(np.int64)


def append(k, v, g, cu, kv, slot_map, k_pages, v_pages, r_pages, carry, PS):
    """Returns (p, k_pages, v_pages, r_pages, carry) as float64 / int64 arrays;
    p is NaN where nothing is written."""
    k, v = f64(k), f64(v)
    e = gate_steps(g)
    T, HQ, K = e.shape
    G = HQ // k.shape[1]
    kp, vp = f64(k_pages), f64(v_pages)
    rp = r_pages.cpu().numpy().astype(np.int64)
    out = carry.cpu().numpy().copy()
    p = np.full((T, HQ, K), np.nan)
    slots = slot_map.cpu().numpy()
    for i in range(len(kv)):
        n = cu[i + 1] - cu[i]
        ctx = kv[i] - n
        if n == 0 or ctx < 0:
            continue
        P = out[i].copy() if ctx > 0 else np.zeros((HQ, K), np.int64)
        for x in range(n):
            t = cu[i] + x
            P = P + e[t]
            page, off = slots[t] // PS, slots[t] % PS
            if (ctx + x) % PS == 0:
                rp[page] = (P + (1 << (FRAC - 1))) >> FRAC
            d = P - (rp[page] << FRAC)
            p[t] = d / float(1 << FRAC)
            kp[page, :, off] = np.repeat(k[t], G, 0) * np.exp2(-p[t])
            vp[page, :, off] = v[t]
        out[i] = P
    return p, kp, vp, rp, out


def attn(q, p, cu, kv, table, k_pages, v_pages, r_pages, PS, scale, sink=None, window=0):
    """(o, lse) float64 of packed rows; NaN past cu[-1]."""
    q, p, kp, vp = f64(q), f64(p), f64(k_pages), f64(v_pages)
    rp = r_pages.cpu().numpy().astype(np.float64)
    table = table.cpu().numpy()
    T, HQ, K = q.shape
    H, V = vp.shape[1], vp.shape[3]
    G = HQ // H
    o = np.full((T, HQ, V), np.nan)
    lse = np.full((T, HQ), np.nan)
    sk = None if sink is None else f64(sink)
    for i in range(len(kv)):
        n = cu[i + 1] - cu[i]
        ctx = kv[i] - n
        for x in range(n):
            t, pos = cu[i] + x, ctx + x
            lo = max(0, pos - window + 1) if window else 0
            js = np.arange(lo, pos + 1) if ctx >= 0 else np.arange(0)
            ids = table[i, js // PS]
            for h in range(HQ):
                if len(js):
                    w = np.exp2(p[t, h] + rp[table[i, pos // PS], h] - rp[ids, h])
                    s = scale * np.einsum("jn,jn->j", w * q[t, h], kp[ids, h, js % PS])
                else:
                    s = np.zeros(0)
                full = s if sk is None else np.append(s, sk[h])
                if len(full) == 0:
                    o[t, h], lse[t, h] = 0.0, -math.inf
                    continue
                m = full.max()
                z = np.exp(full - m).sum()
                lse[t, h] = m + math.log(z)
                o[t, h] = (np.exp(s - m) / z) @ vp[ids, h // G, js % PS] if len(js) else 0.0
    return o, lse
