"""Group norm with an activation on the GPU, forward and backward, against the
FP64 oracle, finite differences and torch.autograd.

Tolerances.  fp32: statistics and sums are fp32 sums of products with rounded
terms (2^-24 each) whose errors grow at most with the depth of the summation
(under 64 sequential additions per thread, then trees): 128 * 2^-24 of the
largest value; sums over rows are held against the sum of their terms'
magnitudes.  bf16 outputs: 2^-8 of the value on top."""
import numpy as np
import pytest
import torch

import gated_delta_rule_157_b200 as kda
from helpers import to_np
from oracle import packed

pytestmark = pytest.mark.gpu
F32 = 128 * 2.0 ** -24


def close(got, want, scale=None):
    step = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    want = np.asarray(want)
    err = np.abs(to_np(got) - want)
    allowed = step * np.abs(want) + F32 * (np.max(np.abs(want)) if scale is None else scale)
    assert np.all(err <= allowed), "%.3g off where %.3g is allowed" % (err.flat[np.argmax(err - allowed)],
                                                                     allowed.flat[np.argmax(err - allowed)])


def inputs(dev, N, L, C, dtype, gated, params=True, seed=0, mean=0.5, shift=0):
    gen = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16

    def act(t):       # `shift` elements off the start of its storage
        flat = torch.empty(t.numel() + shift, dtype=dt, device=dev)[shift:]
        return flat.copy_(t.reshape(-1).to(dt)).view(N, L, C)

    x = act(torch.randn(N, L, C, generator=gen) * 1.5 + mean)
    dy = act(torch.randn(N, L, C, generator=gen))
    z = act(torch.randn(N, L, C, generator=gen)) if gated else None
    w = (1 + 0.3 * torch.randn(C, generator=gen)).to(dev) if params else None
    b = (0.3 * torch.randn(C, generator=gen)).to(dev) if params else None
    return x, dy, z, w, b


def opt(t):
    return None if t is None else to_np(t)


CASES = {
    "token": dict(N=33, L=1, C=512, G=4, dtype="bf16", act="silu", gated=True),
    "token_f32": dict(N=7, L=1, C=320, G=5, dtype="f32", act="sigmoid", gated=False),
    "one_row_one_group": dict(N=1, L=1, C=128, G=1, dtype="bf16", act="none", gated=False),
    "one_channel": dict(N=3, L=1, C=6, G=6, dtype="f32", act="silu", gated=False),
    "odd_width": dict(N=5, L=1, C=21, G=3, dtype="bf16", act="silu", gated=True),
    "wide": dict(N=3, L=1, C=6000, G=1, dtype="bf16", act="none", gated=True),
    "very_wide": dict(N=2, L=1, C=20000, G=2, dtype="f32", act="silu", gated=False),
    "unaligned": dict(N=9, L=1, C=256, G=2, dtype="bf16", act="silu", gated=True, shift=1),
    "many": dict(N=3000, L=1, C=256, G=16, dtype="bf16", act="silu", gated=True),
    "rows": dict(N=2, L=1037, C=320, G=32, dtype="f32", act="silu", gated=False),
    "rows_bf16": dict(N=3, L=515, C=192, G=8, dtype="bf16", act="silu", gated=True),
    "rows_odd": dict(N=2, L=77, C=30, G=10, dtype="bf16", act="sigmoid", gated=False),
    "two_rows": dict(N=4, L=2, C=64, G=2, dtype="f32", act="none", gated=False),
    "rows_unaligned": dict(N=2, L=100, C=64, G=4, dtype="f32", act="silu", gated=True, shift=1),
    "rows_no_params": dict(N=2, L=300, C=64, G=4, dtype="bf16", act="silu", gated=False, params=False),
    "rows_wide": dict(N=1, L=70, C=2304, G=3, dtype="f32", act="silu", gated=False),
}


@pytest.mark.parametrize("name", CASES)
def test_group_norm(cuda_device, name):
    c = dict(CASES[name])
    G, act = c.pop("G"), c.pop("act")
    x, dy, z, w, b = inputs(cuda_device, **c)
    y, mean, rstd = kda.kda_group_norm_fwd(x, G, w, b, z, act=act)
    wy, wm, wr = packed.group_norm(to_np(x), G, opt(w), opt(b), opt(z), act)
    close(y, wy)
    close(mean, wm, np.abs(to_np(x)).max())
    close(rstd, wr)
    d = kda.kda_group_norm_bwd(dy, x, G, mean, rstd, w, b, z, act=act)
    g = packed.group_norm_backward(to_np(dy), to_np(x), G, opt(w), opt(b), opt(z), act)
    # one channel a group: dh cancels to nothing, the error is that of its terms
    close(d["dx"], g["dx"], max(np.abs(g["dx"]).max(), np.abs(to_np(dy)).max() * wr.max()))
    if z is None:
        assert d["dgate"] is None
    else:
        close(d["dgate"], g["dgate"])
    if w is None:
        assert d["dweight"] is None and d["dbias"] is None
    else:
        close(d["dweight"], g["dweight"], g["l1"].max())
        close(d["dbias"], g["dbias"], g["l1"].max())


def test_large_mean_keeps_its_digits(cuda_device):
    """A mean of a thousand standard deviations: the variance is summed about
    the mean, not from squares."""
    for L, C in ((1, 512), (900, 64)):
        x, _, _, w, b = inputs(cuda_device, 3, L, C, "f32", False, mean=1500.0)
        y, mean, rstd = kda.kda_group_norm_fwd(x, 4, w, b)
        wy, wm, wr = packed.group_norm(to_np(x), 4, to_np(w), to_np(b))
        close(mean, wm)
        close(rstd, wr)
        # x itself has 2^-24 * 1500 to spare against a deviation of 1.5: 1000 steps
        assert np.abs(to_np(y) - wy).max() <= 1000 * F32 * np.abs(wy).max()


def test_constant_group_and_eps(cuda_device):
    """A group of one value has variance 0: rstd = eps^-1/2, y = act(bias)."""
    for L in (1, 600):
        x = torch.full((2, L, 64), 3.25, device=cuda_device)
        b = torch.linspace(-1, 1, 64, device=cuda_device)
        y, mean, rstd = kda.kda_group_norm_fwd(x, 4, None, b, act="silu", eps=1e-4)
        assert torch.equal(mean, torch.full_like(mean, 3.25))
        close(rstd, np.full((2, 4), 100.0))
        close(y, np.broadcast_to(to_np(b) / (1 + np.exp(-to_np(b))), (2, L, 64)))


def test_extreme_activations(cuda_device):
    """Gates far out on both sides: no overflow, no NaN; NaN stays in its slab."""
    x, dy, z, w, b = inputs(cuda_device, 4, 1, 256, "f32", True)
    z[0], z[1] = 1e4, -1e4
    z[2] = float("-inf")
    x[3, 0, :128] = float("nan")
    y, mean, rstd = kda.kda_group_norm_fwd(x, 2, w, b, z, act="sigmoid")
    assert torch.isfinite(y[:3]).all() and (y[1:3] == 0).all()
    assert torch.isnan(y[3, 0, :128]).all() and torch.isfinite(y[3, 0, 128:]).all()
    u = packed.group_norm(to_np(x[:1]), 2, to_np(w), to_np(b))[0]
    close(y[:1], u)


@pytest.mark.parametrize("L", [1, 40])
@pytest.mark.parametrize("gated", [False, True])
def test_autograd_against_differences(cuda_device, L, gated):
    """The gradient of <dy, y> through torch.autograd against central
    differences of the FP64 formula in random directions."""
    x, dy, z, w, b = inputs(cuda_device, 2, L, 48, "f32", gated, seed=3)
    leaves = [t.clone().requires_grad_() for t in ([x, w, b] + ([z] if gated else []))]
    y = kda.kda_group_norm(leaves[0], 4, leaves[1], leaves[2], leaves[3] if gated else None, act="silu")
    y.backward(dy)
    gen = np.random.default_rng(0)
    host = [to_np(t) for t in leaves]

    def loss(vals):
        return float((packed.group_norm(vals[0], 4, vals[1], vals[2], vals[3] if gated else None, "silu")[0]
                      * to_np(dy)).sum())

    for i, leaf in enumerate(leaves):
        d = gen.standard_normal(host[i].shape)
        h = 1e-5
        plus, minus = list(host), list(host)
        plus[i], minus[i] = host[i] + h * d, host[i] - h * d
        want = (loss(plus) - loss(minus)) / (2 * h)
        got = float((to_np(leaf.grad) * d).sum())
        # fp32 gradients, summed over all elements, and the difference's own h^2 term
        scale = float((np.abs(to_np(leaf.grad)) * np.abs(d)).sum())
        assert abs(got - want) <= F32 * scale + 1e-8 * scale + 1e-9


def test_autograd_partial_leaves(cuda_device):
    """Only what needs a gradient gets one; a bf16 incoming gradient in fp32 and
    a strided one are taken."""
    x, dy, z, w, b = inputs(cuda_device, 3, 1, 256, "bf16", True)
    w.requires_grad_()
    y = kda.kda_group_norm(x, 2, w, b, z, act="silu")
    y.backward(dy.expand_as(y))
    assert x.grad is None and b.grad is None and w.grad.dtype == torch.float32
    x2 = x.clone().requires_grad_()
    kda.kda_group_norm(x2, 2, act="none").float().sum().backward()
    assert x2.grad.dtype == torch.bfloat16 and x2.grad.abs().max() < 1e-2      # the sum of h is 0


def test_bits_repeat(cuda_device):
    """No atomics: the same bits every run."""
    for L, C in ((1, 1024), (700, 96)):
        x, dy, z, w, b = inputs(cuda_device, 40 if L == 1 else 3, L, C, "bf16", True)
        runs = []
        for _ in range(3):
            y, m, r = kda.kda_group_norm_fwd(x, 4, w, b, z, act="silu")
            d = kda.kda_group_norm_bwd(dy, x, 4, m, r, w, b, z, act="silu")
            runs.append([y, m, r, d["dx"], d["dgate"], d["dweight"], d["dbias"]])
        for other in runs[1:]:
            assert all(torch.equal(a, b_) for a, b_ in zip(runs[0], other))


def test_capture_replay_and_streams(cuda_device):
    """Captured forward and backward replay on new values while an eager graph
    of the same leaves lives; a call on another stream."""
    x, dy, z, w, b = inputs(cuda_device, 3, 300, 64, "bf16", True)
    y, m, r = kda.kda_group_norm_fwd(x, 4, w, b, z, act="silu")
    kda.kda_group_norm_bwd(dy, x, 4, m, r, w, b, z, act="silu")
    eager = kda.kda_group_norm(x.clone().requires_grad_(), 4, w, b, z.clone(), act="silu")   # kept alive
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, m, r = kda.kda_group_norm_fwd(x, 4, w, b, z, act="silu")
        d = kda.kda_group_norm_bwd(dy, x, 4, m, r, w, b, z, act="silu")
    x2, dy2, z2, _, _ = inputs(cuda_device, 3, 300, 64, "bf16", True, seed=8)
    for a, c in ((x, x2), (dy, dy2), (z, z2)):
        a.copy_(c)
    graph.replay()
    close(y, packed.group_norm(to_np(x), 4, to_np(w), to_np(b), to_np(z), "silu")[0])
    g = packed.group_norm_backward(to_np(dy), to_np(x), 4, to_np(w), to_np(b), to_np(z), "silu")
    close(d["dx"], g["dx"])
    close(d["dweight"], g["dweight"], g["l1"].max())
    eager.sum().backward()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, _, _ = kda.kda_group_norm_fwd(x, 4, w, b, z, act="silu")
    s.synchronize()
    assert torch.equal(y, y2)


def test_empty_batch(cuda_device):
    x = torch.empty(0, 5, 64, device=cuda_device)
    w = torch.ones(64, device=cuda_device)
    y, m, r = kda.kda_group_norm_fwd(x, 4, w, w)
    assert y.shape == x.shape and m.shape == (0, 4)
    d = kda.kda_group_norm_bwd(x, x, 4, m, r, w, w)
    torch.cuda.synchronize()
    assert (d["dweight"] == 0).all() and (d["dbias"] == 0).all()


def test_given_stream_owns_what_is_allocated(cuda_device):
    """stream= runs the call, its outputs and its workspace on that stream, with
    the current stream busy over memory that it has just freed."""
    x, dy, z, w, b = inputs(cuda_device, 3, 900, 128, "bf16", True)
    want = packed.group_norm(to_np(x), 4, to_np(w), to_np(b), to_np(z), "silu")[0]
    g = packed.group_norm_backward(to_np(dy), to_np(x), 4, to_np(w), to_np(b), to_np(z), "silu")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        junk = [torch.full((3, 900, 128), float(i), device=cuda_device) for i in range(8)]
        del junk
        y, m, r = kda.kda_group_norm_fwd(x, 4, w, b, z, act="silu", stream=s)
        d = kda.kda_group_norm_bwd(dy, x, 4, m, r, w, b, z, act="silu", stream=s)
        junk = [torch.full((3, 900, 128), float(i), device=cuda_device) for i in range(8)]
        s.synchronize()
        close(y, want)
        close(d["dx"], g["dx"])
        close(d["dweight"], g["dweight"], g["l1"].max())
