"""The direct calls: the ordinary call goes through them and gives the bits of
the Python path (which an explicit output takes); others are left to it."""
import pytest
import torch

import state_space_model_selective_amd as ssm
from state_space_model_selective_amd import hybrid

pytestmark = pytest.mark.gpu
f32, bf16 = torch.float32, torch.bfloat16


def r(*shape, dtype=bf16):
    return torch.randn(*shape, device="cuda").to(dtype)


@pytest.fixture(scope="module")
def fast():
    fast = hybrid._load_fast()
    assert fast.__name__.endswith("_fast_calls"), "the extension is not built"
    return fast


@pytest.mark.parametrize("dtype", [f32, bf16])
def test_same_as_the_python_path(fast, dtype):
    x, gr, gi, A, h = r(2, 300, 66, dtype=dtype), r(2, 300, 66, dtype=dtype), r(2, 300, 66, dtype=dtype), -r(66, dtype=f32).abs(), r(2, 66, dtype=f32)
    last, ck = torch.empty_like(h), torch.empty(ssm.ssm_glr_ckpt_shape(2, 300, 66), device="cuda")
    direct = fast.glr_fwd(x, gr, gi, A, None, last, ck, h, None, None)
    last2, ck2 = torch.empty_like(h), torch.empty_like(ck)
    assert torch.equal(direct, ssm.ssm_glr_fwd(x, gr, gi, A, h0=h, h_last=last2, ckpt=ck2, y=torch.empty_like(x)))
    assert torch.equal(last, last2) and torch.equal(ck, ck2)
    one = [t[:, 0].contiguous() for t in (x, gr, gi)]
    y, h2 = fast.glr_step(*one, A, h, None, None, None)
    y3, h3 = ssm.ssm_glr_step(*one, A, h, y=torch.empty_like(y))
    assert torch.equal(y, y3) and torch.equal(h2, h3)

    packed = r(2, 40, 8, 64, dtype=dtype)
    q, k, v = packed[:, :, :4], packed[:, :, 4:6], packed[:, :, 6:]
    w, freq = r(64, dtype=f32), torch.rand(32, device="cuda", dtype=torch.float64)
    qo, ko = fast.rope_fwd(q, k, w, None, freq, None, 1e-6, None, None, None)
    q2, k2 = ssm.ssm_qk_rope_fwd(q, k, w, None, freq, q_out=torch.empty_like(qo))
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    pos = torch.tensor([5, 100], dtype=torch.int32, device="cuda")
    kc, vc = r(2, 2, 50, 64, dtype=dtype), r(2, 2, 50, 64, dtype=dtype)
    kc2, vc2 = kc.clone(), vc.clone()
    qa = fast.rope_append(q, k, v, w, w, freq, pos, kc, vc, 3, 1e-6, None, None)
    qb = ssm.ssm_qk_rope_append(q, k, v, w, w, freq, pos, kc2, vc2, 3, q_out=torch.empty_like(qa))
    assert torch.equal(qa, qb) and torch.equal(kc, kc2) and torch.equal(vc, vc2)

    lens, lse = torch.tensor([40, 7], dtype=torch.int32, device="cuda"), torch.empty(2, 4, 40, device="cuda")
    o = fast.swa_fwd(qo, k, v, 9, 2, None, lens, None, lse, None)
    lse2 = torch.empty_like(lse)
    assert torch.equal(o, ssm.ssm_swa_fwd(qo, k, v, 9, 2, lens=lens, lse=lse2, o=torch.empty_like(o))) and torch.equal(lse, lse2)
    o = fast.swa_decode(qo[:, 3], kc, vc, pos, None, None, None, None)
    assert torch.equal(o, ssm.ssm_swa_decode(qo[:, 3], kc, vc, pos, o=torch.empty_like(o)))


def test_other_calls_are_left_to_the_python_path(fast):
    x, A, h = r(2, 8), -torch.ones(8, device="cuda"), r(2, 8, dtype=f32)
    ok = (x, x, x, A, h, None, None, None)
    assert fast.glr_step(*ok) is not None
    for i, bad in ((0, x.half()), (1, r(2, 9)), (1, None), (2, r(8, 2).t()), (3, A.cpu()), (3, A.double()), (4, x),
                   (5, x), (6, h), (7, torch.cuda.current_stream()), (0, 3), (4, r(3, 8, dtype=f32))):
        a = list(ok)
        a[i] = bad
        assert fast.glr_step(*a) is None, i
    assert fast.glr_step(*ok[:-1]) is None
    q, k = r(2, 5, 4, 64), r(2, 5, 2, 64)
    ok = (q, k, k, 4, 1, None, None, None, None, None)
    assert fast.swa_fwd(*ok) is not None
    # what the library refuses is refused with its message by the Python path
    for i, bad in ((3, 0), (4, -1), (3, 2.5), (5, -1.0), (0, q[:, :, :3]), (1, k[..., :32]), (2, k[:, :4]), (3, 1 << 70),
                   (0, q.transpose(2, 3)), (6, torch.ones(2, device="cuda"))):
        a = list(ok)
        a[i] = bad
        assert fast.swa_fwd(*a) is None, i
    with pytest.raises(ValueError, match="window"):
        ssm.ssm_swa_fwd(q, k, k, 0)
    with pytest.raises(ssm.SSMError) as e:
        ssm.ssm_swa_fwd(q, k, k, 4, scale=-1.0)
    assert e.value.status == ssm.SSM_ERR_ARG
