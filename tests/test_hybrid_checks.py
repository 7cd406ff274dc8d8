"""Refusals of the hybrid block's entry points, without a GPU: the binding on
CPU tensors, the C ABI on fake addresses that must fail before any HIP call."""
import ctypes
import os
import re

import pytest
import torch

import state_space_model_selective_amd as ssm
from state_space_model_selective_amd import hybrid
from hybrid_util import glr_inputs, glr_reference

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ssm_hybrid.h")
f32, bf16 = torch.float32, torch.bfloat16

# (fake addresses: skipped where a gap in the checks could reach a GPU)
host_only = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="calls the library with fake device addresses")
P = [0x10000000 * (i + 1) for i in range(24)]


def test_every_declared_function_is_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(ssm_[a-z0-9_]+)\s*\(", text))
    assert names == set(hybrid.PROTOTYPES)
    lib = ctypes.CDLL(ssm.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def refuses(match, fn, *a, **kw):
    with pytest.raises((TypeError, ValueError), match=match):
        fn(*a, **kw)


def gpu_only(fn, *a, **kw):
    with pytest.raises(RuntimeError, match="GPU only"):
        fn(*a, **kw)


# --- gated linear recurrence -------------------------------------------------
def glr(dtype=f32):
    t = glr_inputs(2, 20, 6, dtype, seed=0)
    return {k: t[k] for k in ("x", "gr", "gi", "A")}, t


@pytest.mark.parametrize("dtype", [f32, bf16])
def test_glr_valid_arguments_reach_the_gpu_check(dtype):
    a, t = glr(dtype)
    ck = torch.empty(ssm.ssm_glr_ckpt_shape(2, 20, 6))
    assert ck.shape == (2, 2, 6)
    gpu_only(ssm.ssm_glr_fwd, **a, h0=t["h0"], h_last=torch.empty(2, 6), ckpt=ck, y=torch.empty(2, 20, 6, dtype=dtype))
    gpu_only(ssm.ssm_glr_bwd, **a, ckpt=ck, dy=t["dy"], dh_last=t["dh_last"], out={"dA": torch.empty(6)})
    one = {k: v[:, 0].contiguous() if v.dim() == 3 else v for k, v in a.items()}
    gpu_only(ssm.ssm_glr_step, **one, h=t["h0"])


@pytest.mark.parametrize("name,bad", [
    ("x", torch.zeros(2, 20, 6, dtype=torch.float16)), ("x", torch.zeros(20, 6)), ("x", None),
    ("gr", torch.zeros(2, 20, 6, dtype=bf16)), ("gr", torch.zeros(2, 20, 5)), ("gi", torch.zeros(2, 6, 20).transpose(1, 2)),
    ("gi", None), ("A", torch.zeros(6, dtype=torch.float64)), ("A", torch.zeros(5)), ("A", torch.zeros(12)[::2]),
    ("h0", torch.zeros(2, 7)), ("h0", torch.zeros(2, 6, dtype=bf16)), ("y", torch.zeros(2, 20, 6, dtype=bf16)),
    ("h_last", torch.zeros(6, 2)), ("ckpt", torch.zeros(2, 1, 6)), ("gr", torch.zeros(2, 20, 6, device="meta")),
    ("workspace", 3), ("workspace", torch.zeros(4, device="meta"))])
def test_glr_forward_refusals(name, bad):
    a, _ = glr()
    a[name] = bad
    # (the workspace is looked at when its size is known, after the GPU check)
    if name == "workspace":
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            ssm.ssm_glr_fwd(**a)
    else:
        refuses(name, ssm.ssm_glr_fwd, **a)


def test_glr_backward_refusals():
    a, t = glr()
    ck = torch.empty(2, 2, 6)
    refuses("ckpt", ssm.ssm_glr_bwd, **a, ckpt=None, dy=t["dy"])
    refuses("ckpt", ssm.ssm_glr_bwd, **a, ckpt=ck[:, :1], dy=t["dy"])
    refuses("dy", ssm.ssm_glr_bwd, **a, ckpt=ck, dy=t["dy"].to(bf16))
    refuses("dh_last", ssm.ssm_glr_bwd, **a, ckpt=ck, dy=t["dy"], dh_last=torch.zeros(2, 5))
    refuses("unknown output", ssm.ssm_glr_bwd, **a, ckpt=ck, dy=t["dy"], out={"dB": ck})
    refuses("dgr", ssm.ssm_glr_bwd, **a, ckpt=ck, dy=t["dy"], out={"dgr": torch.zeros(2, 20, 6, dtype=bf16)})


def test_glr_step_refusals():
    a, t = glr()
    refuses("x", ssm.ssm_glr_step, **a, h=t["h0"])  # three dimensions
    one = {k: v[:, 0].contiguous() if v.dim() == 3 else v for k, v in a.items()}
    refuses("h ", ssm.ssm_glr_step, **one, h=torch.zeros(2, 6, dtype=bf16))
    refuses("h_out", ssm.ssm_glr_step, **one, h=t["h0"], h_out=torch.zeros(2, 5))


def c_glr_fwd(**kw):
    v = dict(x=P[0], gr=P[1], gi=P[2], A=P[3], h0=P[4], y=P[5], h=P[6], ck=P[7], Bs=2, L=64, ED=64, dt=0, ws=P[8], wb=1 << 30)
    v.update(kw)
    return ssm.lib().ssm_glr_fwd(v["x"], v["gr"], v["gi"], v["A"], v["h0"], v["y"], v["h"], v["ck"], v["Bs"], v["L"],
                                 v["ED"], v["dt"], v["ws"], v["wb"], None)


def c_glr_bwd(**kw):
    v = dict(x=P[0], gr=P[1], gi=P[2], A=P[3], ck=P[4], dy=P[5], dhl=P[6], dx=P[7], dgr=P[8], dgi=P[9], dA=P[10],
             dh0=P[11], Bs=2, L=64, ED=64, dt=0, ws=P[12], wb=1 << 30)
    v.update(kw)
    return ssm.lib().ssm_glr_bwd(*(v[n] for n in ("x", "gr", "gi", "A", "ck", "dy", "dhl", "dx", "dgr", "dgi", "dA",
                                                  "dh0", "Bs", "L", "ED", "dt", "ws", "wb")), None)


def c_glr_step(**kw):
    v = dict(x=P[0], gr=P[1], gi=P[2], A=P[3], h=P[4], y=P[5], ho=P[6], Bs=2, ED=64, dt=0)
    v.update(kw)
    return ssm.lib().ssm_glr_step(*(v[n] for n in ("x", "gr", "gi", "A", "h", "y", "ho", "Bs", "ED", "dt")), None)


@host_only
def test_glr_abi_refusals():
    for n in ("x", "gr", "gi", "A", "y"):
        assert c_glr_fwd(**{n: None}) == ssm.SSM_ERR_NULL
    for n in ("x", "A", "h0", "y", "h", "ck", "ws"):
        assert c_glr_fwd(**{n: P[20] + 4}) == ssm.SSM_ERR_UNSUPPORTED
    for n in ("Bs", "L", "ED"):
        assert c_glr_fwd(**{n: -1}) == ssm.SSM_ERR_DIM
    assert c_glr_fwd(Bs=1 << 40, L=1 << 20, ED=1 << 10) == ssm.SSM_ERR_DIM
    assert c_glr_fwd(dt=2) == ssm.SSM_ERR_UNSUPPORTED
    assert c_glr_fwd(y=P[0]) == ssm.SSM_ERR_ALIAS
    assert c_glr_fwd(ck=P[6] + 64) == ssm.SSM_ERR_ALIAS
    assert c_glr_fwd(h=P[4]) == ssm.SSM_ERR_ALIAS
    assert ssm.ssm_glr_workspace_bytes(1, 4096, 64) > 0
    assert c_glr_fwd(Bs=1, L=4096, ws=None) == ssm.SSM_ERR_WORKSPACE
    assert c_glr_fwd(Bs=1, L=4096, wb=16) == ssm.SSM_ERR_WORKSPACE
    assert c_glr_fwd(Bs=1, L=4096, ws=P[0]) == ssm.SSM_ERR_ALIAS
    for n in ("x", "gr", "gi", "A", "ck", "dy", "dx", "dgr", "dgi", "dA"):
        assert c_glr_bwd(**{n: None}) == ssm.SSM_ERR_NULL
    assert c_glr_bwd(dx=P[1]) == ssm.SSM_ERR_ALIAS
    assert c_glr_bwd(dgi=P[8]) == ssm.SSM_ERR_ALIAS
    assert c_glr_bwd(dh0=P[6]) == ssm.SSM_ERR_ALIAS
    assert c_glr_bwd(ws=None) == ssm.SSM_ERR_WORKSPACE
    assert c_glr_bwd(wb=ssm.ssm_glr_bwd_workspace_bytes(2, 64, 64) - 1) == ssm.SSM_ERR_WORKSPACE
    for n in ("x", "gr", "gi", "A", "h", "y", "ho"):
        assert c_glr_step(**{n: None}) == ssm.SSM_ERR_NULL
    assert c_glr_step(ho=P[4] + 16) == ssm.SSM_ERR_ALIAS
    assert c_glr_step(y=P[4]) == ssm.SSM_ERR_ALIAS
    assert c_glr_step(ED=-1) == ssm.SSM_ERR_DIM
    assert c_glr_step(Bs=0, x=None, gr=None, gi=None, h=None, y=None, ho=None) == ssm.SSM_OK
    assert c_glr_fwd(Bs=0, x=None, gr=None, gi=None, h0=None, y=None, h=None, ck=None) == ssm.SSM_OK
    for bad in ((-1, 2, 3), (1 << 40, 1 << 20, 1 << 10)):
        assert ssm.ssm_glr_workspace_bytes(*bad) == 0 and ssm.ssm_glr_bwd_workspace_bytes(*bad) == 0


def test_glr_reference_gradient():
    """The formula's gradients are those of the recurrence (64-bit differentiation through the loop)."""
    t = {k: v.double() for k, v in glr_inputs(2, 9, 5, f32, seed=1).items()}
    names = ("x", "gr", "gi", "A", "h0")
    leaves = {n: t[n].clone().requires_grad_() for n in names}
    h, loss = leaves["h0"], 0
    for k in range(9):
        a = torch.exp(leaves["A"] * torch.sigmoid(leaves["gr"][:, k]))
        h = a * h + torch.sqrt(1 - a * a) * torch.sigmoid(leaves["gi"][:, k]) * leaves["x"][:, k]
        loss = loss + (h * t["dy"][:, k]).sum()
    loss = loss + (h * t["dh_last"]).sum()
    grads = torch.autograd.grad(loss, [leaves[n] for n in names])
    ref = glr_reference(**t)
    for n, g in zip(names, grads):
        assert torch.allclose(ref["d" + n][0], g, rtol=1e-9, atol=1e-11), n
