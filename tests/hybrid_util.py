"""64-bit definitions of the hybrid block's operators, on the CPU, with the
error that the kernels' roundings can add to each value (test infrastructure).

A rounding to float32 is off by at most EPS = 2^-24 relative to the value; the
constants count how many of them reach a value (each hardware exponential,
reciprocal and square root counts as two, being within one step).
"""
import math

import torch

EPS = torch.finfo(torch.float32).eps / 2


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(name, got, ref, bound):
    """|got - ref| <= bound everywhere (ref finite); says where it is worst."""
    got, ref = got.detach().double().cpu(), ref.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not got.numel():
        return
    assert bool(torch.isfinite(got).all()), "%s: not finite at %s" % (name, (~torch.isfinite(got)).nonzero()[0].tolist())
    over = ((got - ref).abs() - bound).flatten()
    i = int(over.argmax())
    assert float(over[i]) <= 0, "%s: %.9g for %.9g, off by %.3g, allowed %.3g (flat index %d)" % (
        name, got.flatten()[i], ref.flatten()[i], abs(float(got.flatten()[i] - ref.flatten()[i])),
        float(bound.flatten()[i]), i)


def rounded(ref, err, dtype):
    """The error bound of a value stored in dtype: err before the store, then half a step (and the denormal range)."""
    if dtype == torch.float32:
        return err + EPS * ref.abs() + 1e-37
    return err + half_step(dtype) * (ref.abs() + err) + 1e-37


# ---------------------------------------------------------------------------
# gated linear recurrence
# ---------------------------------------------------------------------------
def glr_inputs(Bs, L, ED, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return dict(x=r(Bs, L, ED).to(dtype), gr=(spread * r(Bs, L, ED)).to(dtype), gi=(spread * r(Bs, L, ED)).to(dtype),
                A=-torch.exp(torch.empty(ED).uniform_(math.log(0.004), math.log(2.0), generator=g)),
                h0=r(Bs, ED), dy=r(Bs, L, ED).to(dtype), dh_last=r(Bs, ED))


def glr_reference(x, gr, gi, A, h0=None, dy=None, dh_last=None, **_):
    """{name: (value, error before the store)} of y, h_last and, with dy, the gradients.

    A value of a: the argument A2 r has r's error (2 + 2 + |gr| + 2 roundings,
    times |la|) and its own rounding, the exponential two: 8 + |la| (7 + |gr|).
    A value of s: sqrt halves the relative error of 1 - a^2, which is that of
    la (series, at most 8 roundings) or 2 a^2 / (1 - a^2) < 7 times that of a;
    i has 6 + |gi|, the products two more."""
    x, gr, gi, A = x.double(), gr.double(), gi.double(), A.double()
    Bs, L, ED = x.shape
    h = torch.zeros(Bs, ED, dtype=torch.float64) if h0 is None else h0.double()
    r, i = torch.sigmoid(gr), torch.sigmoid(gi)
    la = A * r
    a, s = la.exp(), (-torch.expm1(2 * la)).clamp(min=0).sqrt()
    ea = EPS * (8 + la.abs() * (7 + gr.abs()))              # relative, of a
    es = EPS * (10 + (7 + gr.abs())) + 4 * ea               # relative, of s
    u = s * i * x
    eu = u.abs() * (es + EPS * (8 + gi.abs()))
    hs, es_h = torch.empty_like(x), torch.empty_like(x)
    h_init, err = h, torch.zeros_like(h)
    for t in range(L):
        new = a[:, t] * h + u[:, t]
        # (the last term: the products of a over a chunk and the joins round a few times more)
        err = a[:, t] * err + (a[:, t] * h.abs()) * (ea[:, t] + 3 * EPS) + eu[:, t] + EPS * new.abs()
        h = new
        hs[:, t], es_h[:, t] = h, err
    out = {"y": (hs, es_h), "h_last": (h, err)}
    if dy is None:
        return out
    dy = dy.double()
    g_all, eg_all = torch.empty_like(x), torch.empty_like(x)
    G = torch.zeros(Bs, ED, dtype=torch.float64) if dh_last is None else dh_last.double()
    eG = torch.zeros_like(G)
    for t in range(L - 1, -1, -1):
        g = dy[:, t] + G
        eg = eG + EPS * g.abs()
        g_all[:, t], eg_all[:, t] = g, eg
        G = a[:, t] * g
        eG = a[:, t] * eg + G.abs() * (ea[:, t] + 3 * EPS)
    hp = torch.cat([h_init.unsqueeze(1), hs[:, :-1]], 1)
    ehp = torch.cat([torch.zeros_like(h_init).unsqueeze(1), es_h[:, :-1]], 1)
    ix, g = i * x, g_all
    root = torch.where(s > 0, a * a / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(s)) * ix
    e_root = root.abs() * (2 * ea + es + EPS * (12 + gi.abs()))
    er = EPS * (6 + gr.abs())
    inner = a * hp - root
    e_inner = a * ehp + (a * hp).abs() * (ea + EPS) + e_root + EPS * inner.abs()
    dlr = g * inner * r
    e_dlr = (eg_all * inner.abs() + g.abs() * e_inner) * r + dlr.abs() * (er + 3 * EPS)
    dx = g * s * i
    dgi = dx * x * (1 - i)
    dgr = dlr * A * (1 - r)
    e_dx = eg_all * s * i + dx.abs() * (es + EPS * (8 + gi.abs()))
    # (1 - i and 1 - r are off by an absolute rounding)
    e_dgi = e_dx * x.abs() * (1 - i) + dgi.abs() * 3 * EPS + (dx * x).abs() * EPS * (7 + gi.abs())
    e_dgr = e_dlr * A.abs() * (1 - r) + dgr.abs() * 3 * EPS + (dlr * A).abs() * EPS * (7 + gr.abs())
    terms = Bs * L
    dA = dlr.sum((0, 1))
    e_dA = e_dlr.sum((0, 1)) + EPS * min(terms, 600) * dlr.abs().sum((0, 1))
    out.update(dx=(dx, e_dx), dgr=(dgr, e_dgr), dgi=(dgi, e_dgi), dA=(dA, e_dA), dh0=(G, eG))
    return out


# ---------------------------------------------------------------------------
# norm and rotation of queries and keys
# ---------------------------------------------------------------------------
def rope_inputs(Bs, L, Hq, Hk, D, R, dtype, seed, far=0):
    """q, k and v are slices of one packed tensor."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    packed = r(Bs, L, Hq + 2 * Hk, D).to(dtype)
    pos = torch.randint(0, far + 1, (Bs, 1), generator=g, dtype=torch.int32) + torch.arange(L, dtype=torch.int32)
    return dict(q=packed[:, :, :Hq], k=packed[:, :, Hq:Hq + Hk], v=packed[:, :, Hq + Hk:], wq=r(D), wk=r(D),
                freq=10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1)), pos=pos,
                dq_out=r(Bs, L, Hq, D).to(dtype), dk_out=r(Bs, L, Hk, D).to(dtype))


def rope_turn(n, pos, freq, back=False):
    R = 2 * freq.numel()
    at = (pos.double().unsqueeze(-1) * freq).unsqueeze(2)
    c, s = at.cos(), at.sin() * (-1 if back else 1)
    a, b = n[..., :R // 2], n[..., R // 2:R]
    return torch.cat([a * c - b * s, b * c + a * s, n[..., R:]], -1)


def rope_reference(x, w, pos, freq, eps, d=None):
    """((value, error), and with d the gradients (dx, error), (dw, error)).

    The mean of squares sums D terms (a butterfly: 8 + 5 roundings), the root
    halves it and adds two; two products: 11 roundings to n. The angle: its
    fraction of a turn is rounded to float32 (half a turn at most: 2 pi EPS / 2
    absolute), the double product is off by 2^-52 of the turns; sine and
    cosine are within 2 EPS: 8 EPS absolute, plus three roundings in the turn."""
    x = x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    inv = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    u = x * inv
    turns = 2.0 ** -51 * float(pos.abs().max()) if pos.numel() else 0.0

    def size(v):  # of a pair, for the errors of its turned values
        R = 2 * freq.numel()
        a, b = v[..., :R // 2].abs(), v[..., R // 2:R].abs()
        return torch.cat([a + b, a + b, v[..., R:].abs()], -1)

    value = rope_turn(u * w, pos, freq)
    err = size(u * w) * (22 * EPS + turns)
    if d is None:
        return value, err
    d = d.double()
    dn, e_dn = rope_turn(d, pos, freq, back=True), size(d) * (11 * EPS + turns)
    t = dn * w
    m = (t * u).mean(-1, keepdim=True)
    e_t = e_dn * w.abs() + EPS * t.abs()
    e_m = (e_t * u.abs() + 24 * EPS * (t * u).abs()).mean(-1, keepdim=True)
    dx = inv * (t - u * m)
    e_dx = inv * (e_t + u.abs() * e_m + (u * m).abs() * 12 * EPS + (t - u * m).abs() * 12 * EPS)
    dw, terms = (dn * u).sum((0, 1, 2)), x[..., 0].numel()
    e_dw = (e_dn * u.abs() + 11 * EPS * (dn * u).abs()).sum((0, 1, 2)) + EPS * min(terms, 1000) * (dn * u).abs().sum((0, 1, 2))
    return (value, err), (dx, e_dx), (dw, e_dw)


# ---------------------------------------------------------------------------
# attention with a sliding window and sinks
# ---------------------------------------------------------------------------
def swa_inputs(Bs, Lq, Lk, Hq, Hk, D, dtype, seed, lens=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype)
    return dict(q=r(Bs, Lq, Hq, D), k=r(Bs, Lk, Hk, D), v=r(Bs, Lk, Hk, D), do=r(Bs, Lq, Hq, D),
                lens=None if lens is None else torch.tensor(lens, dtype=torch.int32))


def swa_seen(Lq, Lk, window, sinks, length):
    p = torch.arange(Lq).unsqueeze(1) + (Lk - Lq)
    j = torch.arange(Lk).unsqueeze(0)
    return (j <= p) & (j < length) & ((p - j < window) | (j < sinks))


def swa_reference(q, k, v, window, sinks, lens=None, do=None, scale=None, rounded_o=None):
    """{name: (value, error before the store)} of o, lse and, with do, dq, dk, dv.

    A score sums D products in float32 (D / 16 steps of an instruction, whose
    own sum counts as one a term: D EPS of the sum of sizes), is multiplied by
    scale log2 e (2) and has the reference point taken off (1). A weight has
    that times ln 2 .. 1 (an absolute error of its exponent), the exponential
    (2), and bfloat16 rounds it by half a step on its way into the product; the
    sums over keys round once a tile at most, counted as Lk of them. delta
    uses the stored o, as the kernel does; lse is stored in float32."""
    dtype = q.dtype
    half = half_step(dtype) if dtype == torch.bfloat16 else 0.0
    Bs, Lq, Hq, D = q.shape
    Lk, Hk = k.shape[1:3]
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64)
    o, eo = z(q), z(q)
    lse, e_lse = (torch.zeros(Bs, Hq, Lq, dtype=torch.float64) for _ in range(2))
    out = {"o": (o, eo), "lse": (lse, e_lse)}
    if do is not None:
        do = do.double()
        out.update(dq=(z(q), z(q)), dk=(z(k), z(k)), dv=(z(v), z(v)))
    for b in range(Bs):
        seen = swa_seen(Lq, Lk, window, sinks, Lk if lens is None else int(lens[b]))
        for h in range(Hq):
            Q, K, V = q[b, :, h], k[b, :, h // G], v[b, :, h // G]
            # unseen keys and values are left out, whatever they hold
            K, V = (torch.where(seen.any(0).unsqueeze(1), t, torch.zeros_like(t)) for t in (K, V))
            s = (Q @ K.T * scale).masked_fill(~seen, -math.inf)
            es = scale * (D + 4) * EPS * (Q.abs() @ K.abs().T) + 4 * EPS * s.masked_fill(~seen, 0).abs()
            L = torch.logsumexp(s, -1)
            some = torch.isfinite(L)
            P = torch.exp(s - torch.where(some, L, torch.zeros_like(L)).unsqueeze(1))
            top = es.masked_fill(~seen, 0).amax(-1, keepdim=True) + 8 * EPS
            ep = P * (es.masked_fill(~seen, 0) + top + 4 * EPS)        # of the unrounded, normalised weight
            sums = (Lk + 8) * EPS
            o[b, :, h] = P @ V
            eo[b, :, h] = (ep + P * (half + sums)) @ V.abs()
            lse[b, h] = L
            e_lse[b, h] = top[:, 0] + sums + 4 * EPS * torch.where(some, L.abs(), torch.zeros_like(L))
            if do is None:
                continue
            dO = do[b, :, h]
            stored = o[b, :, h] if rounded_o is None else rounded_o[b, :, h].double()
            delta = (dO * stored).sum(-1, keepdim=True)
            # (the stored o is the kernel's own, so its error is in delta already; the sum adds D roundings)
            e_delta = D * EPS * (dO * stored).abs().sum(-1, keepdim=True)
            dP = dO @ V.T
            e_dP = (D + 2) * EPS * (dO.abs() @ V.abs().T)
            # lse is stored: another rounding of it reaches the weight
            ep = ep + P * (e_lse[b, h] + EPS * torch.where(some, L.abs(), torch.zeros_like(L))).unsqueeze(1)
            exact_delta = (dO * o[b, :, h]).sum(-1, keepdim=True)
            dS = P * (dP - exact_delta)
            e_ds = ep * (dP - delta).abs() + P * (e_dP + e_delta + (delta - exact_delta).abs()) + 2 * EPS * dS.abs()
            out["dq"][0][b, :, h] = scale * dS @ K
            out["dq"][1][b, :, h] = scale * (e_ds + dS.abs() * (half + sums) + e_ds * half) @ K.abs()
            many = (Lq * G + 8) * EPS
            out["dk"][0][b, :, h // G] += scale * dS.T @ Q
            out["dk"][1][b, :, h // G] += scale * (e_ds + dS.abs() * (half + many) + e_ds * half).T @ Q.abs()
            out["dv"][0][b, :, h // G] += P.T @ dO
            out["dv"][1][b, :, h // G] += (ep + P * (half + many) + ep * half).T @ dO.abs()
    return out
