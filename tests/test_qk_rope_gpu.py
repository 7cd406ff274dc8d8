"""Norm and rotation of queries and keys on the GPU against the 64-bit definition."""
import pytest
import torch

import state_space_model_selective_amd as ssm
from hybrid_util import rope_inputs, rope_reference, rounded, within
from parity_util import log
from test_graph_gpu import replay_check

pytestmark = pytest.mark.gpu

f32, bf16 = torch.float32, torch.bfloat16
EPS = 1e-6
# one token, odd token counts, one to many heads, rotations of the whole head, of parts of it and of nothing
CASES = [(1, 1, 1, 1, 64, 64), (2, 3, 3, 1, 64, 32), (1, 17, 4, 2, 128, 128), (3, 50, 5, 5, 128, 16),
         (1, 1009, 2, 1, 128, 96), (2, 130, 32, 8, 128, 64), (1, 40, 7, 1, 64, 0), (1, 5000, 1, 1, 64, 48)]


def cuda(t):
    """On the GPU, q, k and v again slices of one packed tensor."""
    g = {k: v.cuda() for k, v in t.items() if k not in ("q", "k", "v")}
    packed = torch.cat([t["q"], t["k"], t["v"]], 2).cuda()
    Hq, Hk = t["q"].shape[2], t["k"].shape[2]
    g.update(q=packed[:, :, :Hq], k=packed[:, :, Hq:Hq + Hk], v=packed[:, :, Hq + Hk:])
    if t["freq"].numel() == 0:
        g["freq"] = None
    return g


@pytest.mark.parametrize("dtype", [f32, bf16])
@pytest.mark.parametrize("Bs,L,Hq,Hk,D,R", CASES)
def test_forward_and_gradients(Bs, L, Hq, Hk, D, R, dtype):
    log("qk_rope %d x %d heads %d, %d D %d R %d %s" % (Bs, L, Hq, Hk, D, R, dtype))
    t = rope_inputs(Bs, L, Hq, Hk, D, R, dtype, seed=L + R, far=100)
    g = cuda(t)
    out = dict(zip("qk", ssm.ssm_qk_rope_fwd(g["q"], g["k"], g["wq"], g["wk"], g["freq"], pos=g["pos"], eps=EPS)))
    grads = ssm.ssm_qk_rope_bwd(g["q"], g["k"], g["wq"], g["wk"], g["freq"], g["dq_out"], g["dk_out"], pos=g["pos"], eps=EPS)
    for n in "qk":
        y, dx, dw = rope_reference(t[n], t["w" + n], t["pos"], t["freq"], EPS, t["d%s_out" % n])
        within(n, out[n], y[0], rounded(*y, dtype))
        within("d" + n, grads["d" + n], dx[0], rounded(*dx, dtype))
        within("dw" + n, grads["dw" + n], dw[0], rounded(*dw, f32))


@pytest.mark.parametrize("dtype", [f32, bf16])
def test_far_positions(dtype):
    """Positions near 2^31: the phase is that of the 64-bit product."""
    t = rope_inputs(2, 20, 2, 1, 128, 128, dtype, seed=3)
    t["pos"] = torch.stack([torch.arange(20) + 2 ** 31 - 30, -torch.arange(20) * 10 ** 8]).to(torch.int32)
    g = cuda(t)
    out = ssm.ssm_qk_rope_fwd(g["q"], g["k"], g["wq"], g["wk"], g["freq"], pos=g["pos"], eps=EPS)
    for n, got in zip("qk", out):
        y = rope_reference(t[n], t["w" + n], t["pos"], t["freq"], EPS)
        within(n, got, y[0], rounded(*y, dtype))


def test_without_weights_and_positions():
    t = rope_inputs(2, 30, 4, 2, 64, 64, f32, seed=4)
    t["pos"] = torch.arange(30, dtype=torch.int32).expand(2, 30).contiguous()
    g = cuda(t)
    out = ssm.ssm_qk_rope_fwd(g["q"], g["k"], None, None, g["freq"], eps=EPS)
    grads = ssm.ssm_qk_rope_bwd(g["q"], g["k"], None, g["wk"], g["freq"], g["dq_out"], g["dk_out"], eps=EPS)
    assert sorted(grads) == ["dk", "dq", "dwk"]
    y, dx, _ = rope_reference(t["q"], None, t["pos"], t["freq"], EPS, t["dq_out"])
    within("q", out[0], y[0], rounded(*y, f32))
    within("dq", grads["dq"], dx[0], rounded(*dx, f32))
    _, dx, dw = rope_reference(t["k"], t["wk"], t["pos"], t["freq"], EPS, t["dk_out"])
    within("dk", grads["dk"], dx[0], rounded(*dx, f32))
    within("dwk", grads["dwk"], dw[0], rounded(*dw, f32))


def test_dense_repeated_and_reordered_inputs():
    """Dense tensors, another order of the dimensions in memory, one key head repeated: the same values."""
    t = rope_inputs(2, 21, 4, 1, 64, 64, bf16, seed=5)
    g = cuda(t)
    call = lambda q, k: ssm.ssm_qk_rope_fwd(q, k, g["wq"], g["wk"], g["freq"], pos=g["pos"], eps=EPS)
    q, k = call(g["q"], g["k"])
    dense = call(g["q"].contiguous(), g["k"].contiguous())
    turned = call(g["q"].permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3), g["k"].transpose(1, 2).contiguous().transpose(1, 2))
    for got in (dense, turned):
        assert torch.equal(got[0], q) and torch.equal(got[1], k)
    many = call(g["q"], g["k"].expand(2, 21, 3, 64))[1]
    assert torch.equal(many, k.expand(2, 21, 3, 64))


def test_zero_head_and_non_finite_head():
    """A head of zeros stays zero (eps holds the root); a NaN stays in its head."""
    t = rope_inputs(1, 3, 2, 1, 64, 64, f32, seed=6)
    g = cuda(t)
    g["q"][0, 1, 0] = 0
    want = ssm.ssm_qk_rope_fwd(g["q"], g["k"], g["wq"], g["wk"], g["freq"])
    assert float(want[0][0, 1, 0].abs().max()) == 0
    g["q"][0, 2, 1, 5] = float("nan")
    out = ssm.ssm_qk_rope_fwd(g["q"], g["k"], g["wq"], g["wk"], g["freq"])
    assert bool(torch.isnan(out[0][0, 2, 1]).all())
    out[0][0, 2, 1] = want[0][0, 2, 1]
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def cache_reference(t, g, k_new, k_cache, v_cache, pos, sinks):
    """The cache after the tokens are put one by one."""
    kc, vc, W = k_cache.clone(), v_cache.clone(), k_cache.shape[2] - sinks
    for b, p0 in enumerate(pos.tolist()):
        for l in range(k_new.shape[1] if p0 >= 0 else 0):
            p = p0 + l
            slot = p if p < sinks else sinks + (p - sinks) % W
            kc[b, :, slot], vc[b, :, slot] = k_new[b, l], g["v"][b, l]
    return kc, vc


@pytest.mark.parametrize("dtype", [f32, bf16])
@pytest.mark.parametrize("L,sinks,window", [(1, 4, 16), (1, 0, 1), (7, 2, 5), (40, 3, 8), (5, 0, 64), (33, 4, 16)])
def test_append(L, sinks, window, dtype):
    Bs, Hq, Hk, D = 5, 4, 2, 64
    t = rope_inputs(Bs, L, Hq, Hk, D, 64, dtype, seed=7 + L)
    g = cuda(t)
    pos = torch.tensor([0, 3, -1, window + sinks - 1, 10 ** 6], dtype=torch.int32)
    kc, vc = (torch.randn(Bs, Hk, sinks + window, D, device="cuda").to(dtype) for _ in range(2))
    at = (pos.unsqueeze(1) + torch.arange(L, dtype=torch.int32)).cuda()
    q, k = ssm.ssm_qk_rope_fwd(g["q"], g["k"], g["wq"], g["wk"], g["freq"], pos=at, eps=EPS)
    want_k, want_v = cache_reference(t, g, k, kc, vc, pos, sinks)
    got = ssm.ssm_qk_rope_append(g["q"], g["k"], g["v"], g["wq"], g["wk"], g["freq"], pos.cuda(), kc, vc, sinks, eps=EPS)
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    q[2] = 0  # the inactive row
    assert torch.equal(got, q)


def test_empty():
    z = lambda *s: torch.zeros(*s, device="cuda")
    w, freq = torch.ones(64, device="cuda"), torch.ones(32, device="cuda", dtype=torch.float64)
    for shape in ((0, 4), (2, 0)):
        q, k = ssm.ssm_qk_rope_fwd(z(*shape, 3, 64), z(*shape, 1, 64), w, w, freq)
        assert q.shape == (*shape, 3, 64) and k.shape == (*shape, 1, 64)
        g = ssm.ssm_qk_rope_bwd(z(*shape, 3, 64), z(*shape, 1, 64), w, w, freq, z(*shape, 3, 64), z(*shape, 1, 64))
        assert float(g["dwq"].abs().max()) == 0 and float(g["dwk"].abs().max()) == 0
    q, k = ssm.ssm_qk_rope_fwd(z(2, 4, 0, 64), torch.ones(2, 4, 1, 64, device="cuda"), w, w, freq)
    assert q.shape == (2, 4, 0, 64) and bool((k.abs().sum(-1) > 0).all())


def test_gradient_against_differences():
    t = cuda(rope_inputs(2, 9, 3, 2, 64, 64, f32, seed=8))
    names = ("q", "k", "wq", "wk")
    gen = torch.Generator(device="cuda").manual_seed(3)
    v = {n: torch.randn(t[n].shape, generator=gen, device="cuda") for n in names}

    def loss(step):
        q, k = ssm.ssm_qk_rope_fwd(*(t[n] + step * v[n] for n in names), t["freq"], eps=EPS)
        return float((q.double() * t["dq_out"].double()).sum() + (k.double() * t["dk_out"].double()).sum())

    out = ssm.ssm_qk_rope_bwd(*(t[n] for n in names), t["freq"], t["dq_out"], t["dk_out"], eps=EPS)
    want = sum(float((out["d" + n].double() * v[n].double()).sum()) for n in names)
    eps = 1e-2
    got = (8 * (loss(eps) - loss(-eps)) - (loss(2 * eps) - loss(-2 * eps))) / (12 * eps)
    size = sum(float((out["d" + n].double() * v[n].double()).square().sum()) for n in names) ** 0.5
    assert abs(got - want) <= 1e-3 * size, (got, want, size)


def test_repeated_calls_streams_and_graph():
    g = cuda(rope_inputs(2, 700, 4, 2, 128, 128, bf16, seed=9))
    run = lambda **kw: ssm.ssm_qk_rope_bwd(g["q"], g["k"], g["wq"], g["wk"], g["freq"], g["dq_out"], g["dk_out"],
                                           pos=g["pos"], **kw)
    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = run(stream=side)
    side.synchronize()
    for out in (run(), other):
        for n, v in out.items():
            assert torch.equal(v, first[n]), n
    q, k = ssm.ssm_qk_rope_fwd(g["q"], g["k"], g["wq"], g["wk"], g["freq"], pos=g["pos"])
    grads = {n: torch.empty_like(v) for n, v in first.items()}

    def both():
        ssm.ssm_qk_rope_fwd(g["q"], g["k"], g["wq"], g["wk"], g["freq"], pos=g["pos"], q_out=q, k_out=k)
        run(out=grads)

    replay_check("norm and rotation", both, [q, k] + list(grads.values()))
