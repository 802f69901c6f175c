"""The autograd functions are differentiable once: a second derivative through them
raises instead of losing their terms in silence.  Without a GPU: the library's
calls are replaced by the formulas in torch."""
import pytest
import torch

import gated_delta_rule_157_b200 as kda
from gated_delta_rule_157_b200 import _lib


def _norm(x, groups, weight, bias, gate):
    h = torch.nn.functional.group_norm(x.transpose(1, 2), groups, eps=1e-5).transpose(1, 2)
    return h * weight + bias


@pytest.fixture
def norm_in_torch(monkeypatch):
    def fwd(x, groups, weight=None, bias=None, gate=None, **_):
        stats = torch.zeros(x.shape[0], groups)
        return _norm(x, groups, weight, bias, gate), stats, stats

    def bwd(dy, x, groups, mean, rstd, weight=None, bias=None, gate=None, **_):
        with torch.enable_grad():
            leaves = [t.detach().requires_grad_() for t in (x, weight, bias)]
            got = torch.autograd.grad(_norm(leaves[0], groups, *leaves[1:], gate), leaves, dy)
        return dict(zip(("dx", "dweight", "dbias"), got), dgate=None)

    monkeypatch.setattr(_lib, "kda_group_norm_fwd", fwd)
    monkeypatch.setattr(_lib, "kda_group_norm_bwd", bwd)


def test_group_norm_gradient_has_no_gradient(norm_in_torch):
    x = torch.randn(2, 3, 8, requires_grad=True)
    w, b = torch.ones(8, requires_grad=True), torch.zeros(8, requires_grad=True)
    y = kda.kda_group_norm(x, 2, w, b)
    (dx,) = torch.autograd.grad((y ** 3).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (dx ** 2).sum().backward()
    (y2,) = torch.autograd.grad(kda.kda_group_norm(x, 2, w, b).sum(), x)      # once, as before
    assert y2.shape == x.shape and not y2.requires_grad


def test_chunk_gradient_has_no_gradient(monkeypatch):
    def fwd(q, k, v, *_, **__):
        return v * 2, torch.zeros(v.shape[0], v.shape[2], q.shape[3], v.shape[3]), None

    def bwd(q, k, v, g, beta, S_chunks, do, dS_T, **__):
        return dict(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=do * 2, dg=torch.zeros_like(g),
                    dbeta=torch.zeros_like(beta), dA_log=None, ddt_bias=None, dS0=None)

    monkeypatch.setattr(_lib, "kda_chunk_fwd", fwd)
    monkeypatch.setattr(_lib, "kda_chunk_bwd", bwd)
    q, k, v, g = (torch.randn(1, 4, 1, 8) for _ in range(4))
    v.requires_grad_()
    o, _ = kda.kda_chunk(q, k, v, g, torch.randn(1, 4, 1), gate_in_kernel=False)
    (dv,) = torch.autograd.grad((o ** 3).sum(), v, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (dv ** 2).sum().backward()


def test_packed_calls_refuse_what_needs_a_gradient():
    a, b = torch.zeros(2), torch.zeros(2, requires_grad=True)
    _lib._check_no_grad("call", a, None, a)
    with pytest.raises(ValueError, match="no backward"):
        _lib._check_no_grad("call", a, None, b)
    with torch.no_grad():
        _lib._check_no_grad("call", a, b)
