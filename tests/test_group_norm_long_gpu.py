"""Group norm over many and long slabs on the GPU, against the FP64 formula.

Tolerances.  As in test_group_norm_gpu.py: fp32 statistics and sums, whose errors grow
at most with the depth of the summation, 128 * 2^-24 of the largest value (of the
sum of the terms' magnitudes for the gradients of the parameters).  That depth has
to hold at any length: a slab's rows are summed in short runs, and the runs'
sums in trees."""
import pytest
import torch

import gated_delta_rule_157_b200 as kda

pytestmark = pytest.mark.gpu
F32 = 128 * 2.0 ** -24


def formula(x, G, w, b, dy=None, eps=1e-5):
    """y's statistics, and with dy the gradient of <dy, silu(u)>, in 64 bits on the device."""
    N, L, C = x.shape
    xg = x.double().view(N, L, G, C // G)
    mean = xg.mean((1, 3))
    var = (xg - mean[:, None, :, None]).square().mean((1, 3))
    rstd = (var + eps).rsqrt()
    if dy is None:
        return mean, rstd
    h = ((xg - mean[:, None, :, None]) * rstd[:, None, :, None]).view(N, L, C)
    u = h * w.double() + b.double()
    p = torch.sigmoid(u)
    du = dy.double() * (p * (1 + u * (1 - p)))
    return mean, rstd, (du * h).sum((0, 1)), du.sum((0, 1)), (du * h).abs().sum((0, 1)).max(), du.abs().sum((0, 1)).max()


@pytest.mark.parametrize("N,L,C,G,dtype,sigmas", [
    (256, 4096, 1280, 32, torch.float32, 30.0), (600, 4096, 320, 32, torch.float32, 1000.0),
    (64, 16384, 1024, 32, torch.bfloat16, 1000.0), (3, 1037, 320, 32, torch.float32, 1000.0)])
def test_an_odd_first_row_costs_no_digits(cuda_device, N, L, C, G, dtype, sigmas):
    """The first row of every slab far from the others."""
    gen = torch.Generator(device=cuda_device).manual_seed(1)
    x = torch.randn(N, L, C, generator=gen, device=cuda_device)
    x[:, 0] += sigmas
    x = x.to(dtype)
    _, mean, rstd = kda.kda_group_norm_fwd(x, G)
    for n in range(0, N, 32):
        m, r = formula(x[n:n + 32], G, None, None)
        assert ((rstd[n:n + 32].double() - r).abs() <= F32 * r.max()).all()
        assert ((mean[n:n + 32].double() - m).abs() <= F32 * x[n:n + 32].abs().max().double()).all()


@pytest.mark.parametrize("N,L,C,G,dtype", [(256, 4096, 320, 32, torch.float32), (4, 30000, 1024, 32, torch.bfloat16),
                                           (20000, 3, 64, 4, torch.float32), (200000, 1, 256, 2, torch.bfloat16)])
def test_parameter_gradients_of_many_rows(cuda_device, N, L, C, G, dtype):
    gen = torch.Generator(device=cuda_device).manual_seed(2)
    x = torch.randn(N, L, C, generator=gen, device=cuda_device).add_(0.5).to(dtype)
    dy = torch.randn(N, L, C, generator=gen, device=cuda_device).add_(1.0).to(dtype)
    w = 1 + 0.3 * torch.randn(C, generator=gen, device=cuda_device)
    b = 0.3 * torch.randn(C, generator=gen, device=cuda_device)
    _, mean, rstd = kda.kda_group_norm_fwd(x, G, w, b, act="silu")
    d = kda.kda_group_norm_bwd(dy, x, G, mean, rstd, w, b, act="silu")
    want = [torch.zeros(C, dtype=torch.float64, device=cuda_device) for _ in range(2)]
    l1 = [0.0, 0.0]
    step = max(1, N // 16)
    for n in range(0, N, step):
        got = formula(x[n:n + step], G, w, b, dy[n:n + step])
        for i in range(2):
            want[i] += got[2 + i]
            l1[i] += float(got[4 + i])
    for name, t, s in zip(("dweight", "dbias"), want, l1):
        assert float((d[name].double() - t).abs().max()) <= F32 * s, name


@pytest.mark.parametrize("N,L", [(3, 1), (3, 40), (3, 5000), (700, 1000)])
def test_overflowing_squares_leave_no_small_variance(cuda_device, N, L):
    """Squares beyond the range of fp32: the variance is infinite and rstd 0 in every
    form, and NaN stays NaN."""
    x = torch.randn(N, L, 64, device=cuda_device)
    x[0] = x[0] * 1e30
    x[1, L // 2, 5] = float("nan")
    _, mean, rstd = kda.kda_group_norm_fwd(x, 4)
    assert (rstd[0] == 0).all()
    assert torch.isnan(rstd[1, 0]) and torch.isnan(mean[1, 0])
    m, r = formula(x[2:], 4, None, None)
    assert ((rstd[2:].double() - r).abs() <= F32 * r.max()).all()
    assert torch.isfinite(rstd[1, 1:]).all()


@pytest.mark.parametrize("L", [1, 1500])
def test_parameter_gradients_of_bf16_rows_are_fp32(cuda_device, L):
    """dbias with one term a channel is the activated gate itself: e^-z (1 ulp), 1 + e^-z
    (half), its reciprocal (1) and the sum with zeros -- within 3 * 2^-23 of its value.
    (A sigmoid from a rounded -z log2 e would be off by 2^-18 far out.)"""
    C = 1024
    z = torch.linspace(-86.0, 86.0, C, device=cuda_device).to(torch.bfloat16)
    x = torch.zeros(1, L, C, dtype=torch.bfloat16, device=cuda_device)
    x[0, 0] = 1
    dy = torch.zeros_like(x)
    dy[0, L // 2] = 1
    gate = z.expand(1, L, C).contiguous()
    one, zero = torch.ones(1, 8, device=cuda_device), torch.zeros(1, 8, device=cuda_device)
    w, b = torch.ones(C, device=cuda_device), torch.zeros(C, device=cuda_device)
    d = kda.kda_group_norm_bwd(dy, x, 8, zero, one, w, b, gate, act="sigmoid")
    want = torch.sigmoid(z.double())
    assert float(((d["dbias"].double() - want) / want).abs().max()) <= 3 * 2.0 ** -23
