"""Packed batches on the GPU at their edges: sequences without rows that share a slot,
outputs that the call allocates, bounds that are not what they should be."""
import numpy as np
import pytest
import torch

import gated_delta_rule_157_b200 as kda
from helpers import to_np
from test_packed_gpu import batch, call, check, close, conv_batch, conv_expect, expect

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("per_head,algo", [(False, "auto"), (True, "auto"), (True, "tc"), (True, "simt")])
def test_empty_sequences_may_name_anothers_slot(cuda_device, per_head, algo):
    """A batch padded with empty sequences, ahead of and behind the ones whose slots
    they name: nobody is skipped, nothing is reported."""
    t, kw = batch(cuda_device, [0, 3, 0, 67, 0, 0], 1, 2, 128, 128, "bf16", "softplus", per_head, P=4,
                  slots=[1, 0, 0, 1, 2, 2])
    check(t, kw, algo=algo)            # ends with kda_device_status


def test_empty_sequences_in_the_convolution(cuda_device):
    t, kw = conv_batch(cuda_device, [0, 3, 0, 67, 0, 0], 128, 4, "bf16", slots=[1, 0, 0, 1, 2, 2], P=4)
    y, pool = conv_expect(t, kw)
    kda.kda_packed_conv(t["x"], t["w"], t["pool"], t["bias"], y=t["y"], **kw)
    close(t["y"], y)
    assert np.array_equal(to_np(t["pool"]), pool)
    kda.kda_device_status()


@pytest.mark.parametrize("cu", [[0, 5, 3, 60, 200, 210, 172], [-4, 2, 40, 41, 41, 42, 43], [0, 90, -3, 150, 160, 165, 172]])
def test_convolution_skips_bad_bounds_only(cuda_device, cu):
    """Bounds that run backwards or leave the rows: reported, and every sequence whose
    own bounds are good is computed."""
    t, kw = conv_batch(cuda_device, [3, 70, 4, 50, 2, 40], 256, 4, "bf16", slots=[4, 1, 0, 2, 3, 8], P=9, behind=3)
    kw["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=cuda_device)
    y, pool = conv_expect(t, kw)
    kda.kda_packed_conv(t["x"], t["w"], t["pool"], t["bias"], y=t["y"], **kw)
    assert np.array_equal(to_np(t["pool"]), pool)
    once = torch.ones(172, dtype=torch.bool)
    if cu[1] == 5:                         # rows 3 and 4 are sequence 0's and sequence 2's: either's result
        once[3:5] = False
    close(t["y"][once.to(cuda_device)], y[once.numpy()])
    with pytest.raises(kda.KdaError):
        kda.kda_device_status()


def test_tensors_that_require_grad_are_refused(cuda_device):
    """The packed calls have no backward: every floating tensor is looked at."""
    for name in ("q", "k", "v", "g", "beta", "pool", "A_log", "dt_bias"):
        t, kw = batch(cuda_device, [3, 2], 1, 2, 128, 128, "bf16", "bounded", False)
        (kw if name in kw else t)[name].requires_grad_()
        with pytest.raises(ValueError, match="no backward"):
            call(t, kw)
        with torch.no_grad():
            call(t, kw)
    for name in ("x", "w", "bias", "pool"):
        t, kw = conv_batch(cuda_device, [3, 2], 128, 4, "bf16")
        t[name].requires_grad_()
        with pytest.raises(ValueError, match="no backward"):
            kda.kda_packed_conv(t["x"], t["w"], t["pool"], t["bias"], **kw)
        with torch.no_grad():
            kda.kda_packed_conv(t["x"], t["w"], t["pool"], t["bias"], **kw)


def test_rows_that_are_left_out_of_a_new_output_are_zero(cuda_device):
    """Skipped sequences and rows outside every sequence, where the call allocates
    the output over memory that held something else."""
    for per_head in (False, True):
        t, kw = batch(cuda_device, [3, 20, 40], 1, 2, 128, 128, "bf16", "softplus", per_head, slots=[1, -1, 0], behind=7)
        t["o"].zero_()
        o, _ = expect(t, kw)
        junk = torch.full_like(t["o"], float("nan"))
        del junk
        got = kda.kda_packed_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["pool"], **kw)
        assert (got[3:23] == 0).all() and (got[63:] == 0).all()
        close(got, o)
    t, kw = conv_batch(cuda_device, [4, 5, 6], 128, 4, "bf16", slots=[2, -1, 0], behind=3)
    t["y"].zero_()
    y, _ = conv_expect(t, kw)
    junk = torch.full_like(t["y"], float("nan"))
    del junk
    got = kda.kda_packed_conv(t["x"], t["w"], t["pool"], t["bias"], **kw)
    assert (got[4:9] == 0).all() and (got[15:] == 0).all()
    close(got, y)


@pytest.mark.parametrize("per_head,algo", [(False, "auto"), (True, "tc"), (True, "simt")])
def test_outputs_whose_rows_lie_apart(cuda_device, per_head, algo):
    """o and y as columns of wider rows, whose other columns stay as they were."""
    t, kw = batch(cuda_device, [3, 70, 1], 1, 2, 128, 128, "bf16", "softplus", per_head)
    wide = torch.full((74, 400), 0.0625, dtype=torch.bfloat16, device=cuda_device)
    t["o"] = wide[:, 64:320].unflatten(1, (2, 128))
    check(t, kw, algo=algo)
    assert (wide[:, :64] == 0.0625).all() and (wide[:, 320:] == 0.0625).all()
    t, kw = conv_batch(cuda_device, [3, 70, 1], 256, 4, "bf16")
    wide = torch.full((74, 400), 0.0625, dtype=torch.bfloat16, device=cuda_device)
    y, _ = conv_expect(t, kw)
    kda.kda_packed_conv(t["x"], t["w"], t["pool"], t["bias"], y=wide[:, 64:320], **kw)
    close(wide[:, 64:320], y)
    assert (wide[:, :64] == 0.0625).all() and (wide[:, 320:] == 0.0625).all()


@pytest.mark.parametrize("per_head", [False, True])
def test_bounds_without_slots(cuda_device, per_head):
    """Sequence s has slot s; a pool larger than the batch keeps its other slots."""
    t, kw = batch(cuda_device, [5, 0, 80, 1], 1, 2, 128, 128, "bf16", "softplus", per_head, P=6, slots=[0, 1, 2, 3])
    kw["slots"] = torch.arange(4, dtype=torch.int32, device=cuda_device)
    o, pool = expect(t, kw)
    call(t, dict(kw, slots=None))
    close(t["o"], o)
    close(t["pool"], pool)
    kda.kda_device_status()


def test_no_rows_and_no_sequences(cuda_device):
    """Empty batches change nothing."""
    for lens in ([], [0, 0]):
        t, kw = batch(cuda_device, lens, 1, 2, 128, 128, "bf16", "softplus", True, P=3)
        kw["slots"] = torch.arange(len(lens), dtype=torch.int32, device=cuda_device)
        before = t["pool"].clone()
        for algo in ("auto", "simt", "tc"):
            assert call(t, kw, algo=algo).shape == (0, 2, 128)
        assert torch.equal(t["pool"], before)
        c, ck = conv_batch(cuda_device, lens, 128, 4, "bf16", P=3)
        ck["slots"] = kw["slots"]
        before = c["pool"].clone()
        assert kda.kda_packed_conv(c["x"], c["w"], c["pool"], c["bias"], **ck).shape == (0, 128)
        assert torch.equal(c["pool"], before)
    kda.kda_device_status()


def test_two_captured_calls_share_a_pool(cuda_device):
    """Two graphs over slots of one pool, replayed in turn and on two streams."""
    made = [batch(cuda_device, [70, 2], 1, 2, 128, 128, "bf16", "softplus", True, seed=i, slots=[2 * i, 2 * i + 1], P=4)
            for i in range(2)]
    pool = made[0][0]["pool"]
    made[1][0]["pool"] = pool
    start = pool.clone()
    graphs, outs = [], []
    for t, kw in made:
        call(t, kw)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(kda.kda_packed_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], pool, **kw))
        graphs.append(graph)
    pool.copy_(start)
    want = [expect(t, kw) for t, kw in made]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, graph in zip(streams, graphs):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        close(outs[i], want[i][0])
        close(pool[2 * i:2 * i + 2], want[i][1][2 * i:2 * i + 2])
