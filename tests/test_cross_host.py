"""Host-only checks of cross attention: bad arguments return the documented codes before any GPU is touched,
and the float64 form that the GPU tests compare with agrees with an independent statement of the definition."""
import math
import os
import shutil

import pytest
import torch

import flashattention_backward_fa_gb300 as fa
from flashattention_backward_fa_gb300 import binding
from cross_reference import Reference

F32, F16, BF16 = fa.FA_F32, fa.FA_F16, fa.FA_BF16
EINVAL, EUNSUP, EALIGN, EWS = -1, -2, -3, -4
P = 0x10000  # a fake, 256-byte-aligned "device" address: validation rejects before any use


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("no nvcc to build the library")
        from flashattention_backward_fa_gb300.build import build_library
        build_library()
    return fa.load_library()


def _call(lib, back, *, B=2, Nq=8, Nk=100, Hq=4, Hk=2, d=64, ql=None, kl=None, dt=BF16, scale=0.1, q=P, k=P, v=P, o=P,
          lse=P, g=P, st=None, kst=None, ws=P, size=1 << 40):
    shape = binding._CrossShape(B, Nq, Nk, Hq, Hk, d, ql, kl)
    qs = st or fa.FaStrides(Nq * max(Hq, 1) * d, max(Hq, 1) * d, d)
    ks = kst or fa.FaStrides(Nk * max(Hk, 1) * d, max(Hk, 1) * d, d)
    if back:
        return lib.fa_cross_bwd(shape, q, k, v, o, g, lse, P, P, P, qs, ks, ks, qs, qs, qs, ks, ks, dt, scale, ws, size,
                                None)
    return lib.fa_cross_fwd(shape, q, k, v, o, lse, qs, ks, ks, qs, dt, scale, ws, size, None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(B=0), EINVAL), (dict(Nq=0), EINVAL), (dict(Nk=0), EINVAL), (dict(Hq=0), EINVAL), (dict(Hk=0), EINVAL),
    (dict(d=0), EINVAL), (dict(Hq=3), EINVAL), (dict(Hq=1), EINVAL), (dict(B=-1), EINVAL),
    (dict(dt=3), EUNSUP), (dict(d=96), EUNSUP), (dict(d=129, dt=F32), EUNSUP), (dict(B=65536), EUNSUP),
    (dict(Hq=65536, Hk=1), EUNSUP), (dict(Nq=(1 << 24) + 1), EUNSUP), (dict(Nk=(1 << 24) + 1), EUNSUP),
    (dict(B=60000, Hq=1024), EUNSUP), (dict(Nq=1 << 24, Hq=128, Hk=1), EUNSUP),
    (dict(ql=P + 2), EALIGN), (dict(kl=P + 1), EALIGN),
    (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL), (dict(scale=math.nan), EINVAL), (dict(scale=math.inf), EINVAL),
    (dict(q=0), EINVAL), (dict(k=0), EINVAL), (dict(v=0), EINVAL), (dict(o=0), EINVAL), (dict(lse=0), EINVAL),
    (dict(q=P + 8), EALIGN), (dict(v=P + 2), EALIGN), (dict(o=P + 4), EALIGN), (dict(lse=P + 4), EALIGN),
    (dict(st=fa.FaStrides(4096, 260, 64)), EALIGN), (dict(kst=fa.FaStrides(0, 128, 64)), EINVAL),
    (dict(kst=fa.FaStrides(12800, 128, -64)), EINVAL),
])
def test_rejects_bad_arguments(lib, back, kw, code):
    assert _call(lib, back, **kw) == code


def test_rejects_bad_workspaces(lib):
    split = dict(B=1, Nq=1, Nk=100000, Hq=4, Hk=2)
    need = fa.fa_cross_fwd_workspace_size(1, 1, 100000, 4, 2, 64, torch.bfloat16)
    assert need > 0 and need % 256 == 0
    assert _call(lib, False, **split, ws=0) == EWS
    assert _call(lib, False, **split, ws=P + 128) == EWS
    assert _call(lib, False, **split, size=need - 1) == EWS
    need = fa.fa_cross_bwd_workspace_size(2, 8, 100, 4, 2, 64, torch.bfloat16)
    assert need > 0 and need % 256 == 0
    assert _call(lib, True, ws=0) == EWS
    assert _call(lib, True, ws=P + 64) == EWS
    assert _call(lib, True, size=need - 1) == EWS
    assert _call(lib, True, g=0) == EINVAL


def test_workspace_sizes(lib):
    size = fa.fa_cross_fwd_workspace_size
    assert size(32, 4096, 512, 16, 16, 128, torch.bfloat16) == 0  # enough blocks without splits
    for bad in ((0, 1, 1, 1, 1, 64), (1, 1, 1, 3, 2, 64), (1, 1, 1, 1, 1, 80)):
        assert size(*bad, torch.float16) == 0 and fa.fa_cross_bwd_workspace_size(*bad, torch.float16) == 0
    assert lib.fa_cross_fwd_workspace_size(None, BF16) == 0 and lib.fa_cross_bwd_workspace_size(None, BF16) == 0


def test_host_pointers_are_refused(lib):
    if torch.cuda.is_available():
        pytest.skip("covered on the GPU by the binding's own checks")
    assert _call(lib, False) != 0 and _call(lib, True) != 0


def test_reference_agrees_with_autograd():
    """The loops of the reference against one masked softmax over the whole batch, and its gradients."""
    torch.manual_seed(0)
    B, Nq, Nk, Hq, Hk, d = 3, 5, 7, 4, 2, 16
    q, k, v = (torch.randn(B, n, h, d, dtype=torch.float64) for n, h in ((Nq, Hq), (Nk, Hk), (Nk, Hk)))
    do = torch.randn_like(q)
    ql, kl = torch.tensor([5, 2, 4]), torch.tensor([7, 3, 0])
    for t in (q, k, v):
        t.requires_grad_()
    kk, vv = (t.repeat_interleave(Hq // Hk, 2) for t in (k, v))
    live_q = torch.arange(Nq)[None] < ql[:, None]
    live_k = torch.arange(Nk)[None] < kl[:, None]
    s = torch.einsum("bihd,bjhd->bhij", q, kk) * 0.3
    s = s.masked_fill(~live_k[:, None, None], -1e300)
    p = s.softmax(-1) * live_k[:, None, None] * live_q[:, None, :, None]
    o = torch.einsum("bhij,bjhd->bihd", p, vv)
    grads = torch.autograd.grad(o, (q, k, v), do)
    ref = Reference(q.detach(), k.detach(), v.detach(), ql, kl, 0.3, do)
    for name, a in zip(("o", "dq", "dk", "dv"), (o.detach(),) + grads):
        assert (getattr(ref, name) - a).abs().max() < 1e-12, name
    assert (ref.lse[2] == -math.inf).all() and (ref.lse[1, :, 2:] == -math.inf).all()
    assert torch.allclose(ref.lse[0], (torch.einsum("ihd,jhd->hij", q[0], kk[0]) * 0.3).logsumexp(-1).detach())


def test_binding_refuses_cpu_tensors():
    t = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.cross_attention_forward(t, t, t)
    with pytest.raises(ValueError):
        fa.cross_attn_func(t, t, t)
