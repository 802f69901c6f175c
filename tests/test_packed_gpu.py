"""Packed batches on the GPU (delta rule, short convolution) against the FP64
oracle.

Tolerances.  A rounding is off by at most half a step: 2^-24 of the value in
fp32, 2^-8 in bf16.  An fp32 result is a sum of at most 128 products, each
rounded, with a state that every token contracts and adds one rounded term to:
within 2 * 128 * 2^-24 of the largest value.  A bf16 output is that rounded
once more: 2^-8 of its own value on top.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_157_b200 as kda
from helpers import to_np
from oracle import packed

pytestmark = pytest.mark.gpu
F32 = 256 * 2.0 ** -24


def close(got, want, what=""):
    """Every element within the tolerance of its type."""
    step = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    want = np.asarray(want)
    if want.size == 0:
        return
    err = np.abs(to_np(got) - want)
    allowed = step * np.abs(want) + F32 * np.max(np.abs(want))
    assert np.all(err <= allowed), "%s: %.3g off where %.3g is allowed" % (
        what, err.flat[np.argmax(err - allowed)], allowed.flat[np.argmax(err - allowed)])


def rows(gen, T, shape, dt, pad, dev):
    w = int(np.prod(shape))
    return torch.randn(T, w + pad, generator=gen).to(dt).to(dev)[:, :w].unflatten(1, shape)


def batch(dev, lens, H, HV, Dk, Dv, dtype, gate, per_head, seed=0, pad=0, slots=None, fresh=None, P=None, z_mean=0.0,
          behind=0, scale=0.25):
    """Inputs of a packed call: a dict of tensors and the keyword arguments."""
    gen = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    T, n = sum(lens) + behind, len(lens)
    gk = () if per_head else (Dk,)
    t = {"q": rows(gen, T, (H, Dk), dt, pad, dev), "k": rows(gen, T, (H, Dk), dt, pad, dev),
         "v": rows(gen, T, (HV, Dv), dt, pad, dev), "g": rows(gen, T, (HV,) + gk, dt, pad, dev),
         "beta": rows(gen, T, (HV,), dt, pad, dev)}
    t["g"] += z_mean
    if not gate:
        t["g"] = -t["g"].abs() * 0.3
    P = P or n + 2
    if slots is None:
        slots = torch.randperm(P, generator=gen)[:n].tolist()
    t["pool"] = (torch.randn(P, HV, Dk, Dv, generator=gen) * 0.1).to(dev)
    t["o"] = torch.full((T, HV, Dv), 0.0625, dtype=dt, device=dev)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    A = torch.rand(HV, generator=gen) * 2 - 1
    b = torch.randn((HV,) + gk, generator=gen) * 0.5
    kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev),
              slots=torch.tensor(slots, dtype=torch.int32, device=dev),
              fresh=None if fresh is None else torch.tensor(fresh, dtype=torch.bool, device=dev),
              A_log=A.to(dev), dt_bias=b.to(dev), gate_in_kernel=gate, g_per_head=per_head, scale=scale)
    return t, kw


def call(t, kw, **more):
    return kda.kda_packed_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["pool"], o=t["o"], **kw, **more)


def expect(t, kw):
    """The oracle's (o, pool) from the tensors as they are now."""
    host = lambda x: None if x is None else x.tolist()     # noqa: E731
    return packed.packed_fwd(*(to_np(t[n]) for n in ("q", "k", "v", "g", "beta", "pool", "o")),
                             cu=host(kw["cu_seqlens"]), slots=host(kw["slots"]), fresh=host(kw["fresh"]),
                             A_log=to_np(kw["A_log"]), dt_bias=to_np(kw["dt_bias"]), gate=kw["gate_in_kernel"],
                             per_head=kw["g_per_head"], scale=kw["scale"])


def check(t, kw, **more):
    o, pool = expect(t, kw)
    call(t, kw, **more)
    close(t["o"], o, "o")
    close(t["pool"], pool, "pool")
    kda.kda_device_status()


CASES = {
    # one token each, every type and decay
    "step_bf16": dict(lens=[1] * 9, H=2, HV=4, Dk=128, Dv=128, dtype="bf16", gate="bounded", per_head=False),
    "step_f32_head": dict(lens=[1] * 3, H=1, HV=3, Dk=64, Dv=96, dtype="f32", gate="softplus", per_head=True),
    "step_given_decay": dict(lens=[1, 1], H=1, HV=1, Dk=128, Dv=128, dtype="bf16", gate=False, per_head=False),
    # odd widths, rows that lie apart (also off 16-byte and 4-byte boundaries)
    "odd_f32": dict(lens=[5, 0, 1, 17, 33], H=1, HV=2, Dk=65, Dv=36, dtype="f32", gate="bounded", per_head=False,
                    pad=1),
    "odd_bf16": dict(lens=[2, 9, 40], H=2, HV=2, Dk=1, Dv=4, dtype="bf16", gate="softplus", per_head=True, pad=3),
    "narrow": dict(lens=[7, 8, 9], H=3, HV=3, Dk=17, Dv=12, dtype="bf16", gate="bounded", per_head=False),
    # ragged prefill, some from zero, rows behind the last sequence
    "prefill_f32": dict(lens=[70, 1, 0, 200], H=1, HV=2, Dk=128, Dv=128, dtype="f32", gate="bounded", per_head=False,
                        fresh=[1, 0, 1, 0], behind=5),
    "prefill_bf16": dict(lens=[129, 3, 64], H=2, HV=4, Dk=128, Dv=128, dtype="bf16", gate="softplus", per_head=False,
                         fresh=[0, 1, 1]),
    # decays that reach zero, and none at all
    "strong": dict(lens=[50, 20], H=1, HV=2, Dk=128, Dv=64, dtype="f32", gate="softplus", per_head=False, z_mean=60.0),
    "weak": dict(lens=[50, 20], H=1, HV=2, Dk=128, Dv=64, dtype="f32", gate="softplus", per_head=True, z_mean=-60.0),
}


@pytest.mark.parametrize("name", CASES)
def test_recurrence(cuda_device, name):
    check(*batch(cuda_device, **CASES[name]), algo="simt")


CHUNKS = {
    "one": dict(lens=[1], H=1, HV=1, gate="softplus"),
    "whole_chunk": dict(lens=[64], H=1, HV=1, gate="bounded"),
    "ragged": dict(lens=[65, 0, 63, 200, 1, 129], H=2, HV=4, gate="softplus", fresh=[1, 0, 0, 1, 0, 1], behind=70),
    "given_decay": dict(lens=[130, 40], H=1, HV=2, gate=False),
    "views": dict(lens=[100, 33], H=1, HV=2, gate="softplus", pad=8),
    "strong": dict(lens=[200, 70], H=1, HV=1, gate="softplus", z_mean=60.0),
    "mixed_decay": dict(lens=[300], H=1, HV=2, gate="softplus", z_mean=3.0),
    "weak": dict(lens=[200, 70], H=1, HV=1, gate="softplus", z_mean=-60.0),
    # more chains than CTAs, more sequences than a page of the schedule
    "many_chains": dict(lens=[90, 3, 70, 1, 40] * 3, H=4, HV=16, gate="softplus"),
    "many_sequences": dict(lens=[1, 2, 66] * 200, H=1, HV=1, gate="softplus"),
    "long": dict(lens=[2500], H=1, HV=2, gate="softplus", z_mean=-5.0),
}


@pytest.mark.parametrize("name", CHUNKS)
def test_chunks(cuda_device, name):
    check(*batch(cuda_device, Dk=128, Dv=128, dtype="bf16", per_head=True, **CHUNKS[name]), algo="tc")


@pytest.mark.parametrize("name", ["ragged", "many_chains"])
def test_chunks_and_recurrence_share_a_batch(cuda_device, name):
    """AUTO: the long sequences in chunks, the short ones by the recurrence."""
    check(*batch(cuda_device, Dk=128, Dv=128, dtype="bf16", per_head=True, **CHUNKS[name]))


def test_alike_keys(cuda_device):
    """Every key the same and no decay: the triangular system at its worst
    (T's entries cancel; powers of A would grow to 10^17).

    o is here much smaller than the terms it is the sum of, so its bound is
    theirs: inside a chunk o_i = ... + sum_j B_ij U_j, with B and U as two bf16
    terms each.  Two terms leave 2^-18 of the value, and the product of the two
    tails that is left out is 2^-9 * 2^-9 of it, so each product is off by at
    most 3 * 2^-18 |B_ij U_j|."""
    t, kw = batch(cuda_device, [128], 1, 1, 128, 128, "bf16", "softplus", True, z_mean=-60.0)
    t["k"][:] = t["k"][:1]
    t["beta"][:] = 6.0
    o, pool = expect(t, kw)
    q, k, v = (to_np(t[n])[:, 0] for n in ("q", "k", "v"))
    B = kw["scale"] * np.abs((q / np.linalg.norm(q, axis=1, keepdims=True)) @ (k[0] / np.linalg.norm(k[0])))
    beta = 1 / (1 + np.exp(-6.0))
    y = to_np(t["pool"])[int(kw["slots"][0]), 0].T @ (k[0] / np.linalg.norm(k[0]))      # S^T k
    U = np.empty_like(v)
    for i in range(128):
        U[i] = beta * (v[i] - y)
        y = y + U[i]
    sums = np.stack([np.abs(U[i // 64 * 64: i + 1]).sum(0) * B[i] for i in range(128)])
    call(t, kw, algo="tc")
    err = np.abs(to_np(t["o"])[:, 0] - o[:, 0])
    assert np.all(err <= 2.0 ** -8 * np.abs(o[:, 0]) + F32 * np.abs(o).max() + 3 * 2.0 ** -18 * sums)
    close(t["pool"], pool, "pool")


@pytest.mark.parametrize("name", ["step_bf16", "odd_f32", "prefill_bf16"])
def test_known_longest_length_changes_nothing(cuda_device, name):
    t, kw = batch(cuda_device, **CASES[name])
    u, _ = batch(cuda_device, **CASES[name])
    a = call(t, kw)
    b = call(u, kw, max_seqlen=max(CASES[name]["lens"]))
    assert torch.equal(a, b) and torch.equal(t["pool"], u["pool"])


def test_wrong_longest_length(cuda_device):
    """A longest length given too small costs time, not results."""
    check(*batch(cuda_device, [30, 1, 17, 100], 1, 2, 128, 128, "bf16", "softplus", True), max_seqlen=1)
    check(*batch(cuda_device, [30, 1, 17, 100], 1, 2, 40, 20, "f32", "bounded", False), max_seqlen=2)


@pytest.mark.parametrize("switch", ["qk_l2norm_in_kernel", "beta_sigmoid_in_kernel"])
def test_switches(cuda_device, switch):
    t, kw = batch(cuda_device, [6, 11], 1, 2, 32, 32, "f32", "bounded", False)
    if switch[0] == "q":
        t["q"], t["k"] = t["q"] / 8, t["k"] / 8
    else:
        t["beta"] = torch.sigmoid(t["beta"])
    host = lambda x: None if x is None else x.tolist()     # noqa: E731
    o, pool = packed.packed_fwd(*(to_np(t[n]) for n in ("q", "k", "v", "g", "beta", "pool", "o")),
                                cu=host(kw["cu_seqlens"]), slots=host(kw["slots"]), A_log=to_np(kw["A_log"]),
                                dt_bias=to_np(kw["dt_bias"]), scale=kw["scale"],
                                **{"l2norm" if switch[0] == "q" else "beta_sigmoid": False})
    call(t, kw, **{switch: False})
    close(t["o"], o)
    close(t["pool"], pool)


def test_rows_without_bounds_are_a_step(cuda_device):
    t, kw = batch(cuda_device, [1] * 5, 1, 2, 128, 128, "bf16", "bounded", False)
    u, _ = batch(cuda_device, [1] * 5, 1, 2, 128, 128, "bf16", "bounded", False)
    call(t, kw)
    call(u, dict(kw, cu_seqlens=None))
    assert torch.equal(t["o"], u["o"]) and torch.equal(t["pool"], u["pool"])


def test_equals_the_decode_step(cuda_device):
    """One token each against kda_step on the same states."""
    t, kw = batch(cuda_device, [1] * 6, 2, 4, 128, 128, "bf16", "bounded", False, P=6, slots=list(range(6)))
    S = t["pool"].clone()
    o = kda.kda_step(S, *(t[n] for n in ("q", "k", "v", "g", "beta")), A_log=kw["A_log"], dt_bias=kw["dt_bias"],
                     scale=kw["scale"])
    call(t, kw)
    close(t["o"], to_np(o))            # both rounded: within one step of each other
    close(t["pool"], to_np(S))


@pytest.mark.parametrize("per_head", [False, True])
def test_skipped_sequences(cuda_device, per_head):
    """Slot -1 is skipped in silence; a slot out of the pool, a repeated slot and
    bounds that run backwards or out of range are skipped and reported; rows and
    slots of skipped sequences keep what they hold."""
    t, kw = batch(cuda_device, [3, 70, 4, 50, 2, 40], 1, 2, 128, 128, "bf16", "softplus", per_head, P=9,
                  slots=[4, -1, 0, 4, 9, 8], behind=3)
    o, pool = expect(t, kw)
    call(t, kw)
    close(t["o"], o)
    close(t["pool"], pool)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_device_status()
    assert e.value.status == 7
    kda.kda_device_status()
    untouched = torch.full_like(t["o"][:1], 0.0625)
    assert (t["o"][3:73] == untouched).all() and (t["o"][77:129] == untouched).all()
    for cu in ([0, 5, 3, 60, 200, 210, 172], [-4, 2, 40, 41, 41, 42, 43]):
        t, kw = batch(cuda_device, [3, 70, 4, 50, 2, 40], 1, 2, 128, 128, "bf16", "softplus", per_head, P=9,
                      slots=[4, 1, 0, 2, 3, 8], behind=3)
        kw["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=cuda_device)
        o, pool = expect(t, kw)
        call(t, kw)
        close(t["pool"], pool)
        once = torch.ones(172, dtype=torch.bool)
        if cu[1] > cu[2]:                  # rows 3 and 4 are sequence 0's and sequence 2's: either's result
            once[3:5] = False
        close(t["o"][once.to(cuda_device)], o[once.numpy()])
        with pytest.raises(kda.KdaError):
            kda.kda_device_status()


def test_non_finite_values_stay_in_their_sequence(cuda_device):
    """Infinities and NaN in one request, and in rows that belong to none, reach
    nobody else."""
    for per_head in (False, True):
        t, kw = batch(cuda_device, [40, 70, 33, 2], 1, 2, 128, 128, "bf16", "softplus", per_head, behind=40)
        o, pool = expect(t, kw)
        for n in ("q", "k", "v", "g", "beta"):
            t[n][40:110] = float("nan")
            t[n][145:] = float("inf")
        call(t, kw)
        keep = torch.ones(t["o"].shape[0], dtype=torch.bool)
        keep[40:110] = False
        close(t["o"][keep.to(cuda_device)], o[keep.numpy()])
        for s in (0, 2, 3):
            slot = int(kw["slots"][s])
            close(t["pool"][slot], pool[slot])


def test_fresh_ignores_what_the_slot_holds(cuda_device):
    for lens in ([4, 40], [40, 90]):
        t, kw = batch(cuda_device, lens, 1, 1, 128, 128, "bf16", "softplus", True, fresh=[1, 1])
        o, pool = expect(t, kw)
        for s in range(2):
            t["pool"][int(kw["slots"][s])] = float("nan")
        call(t, kw)
        close(t["o"], o)
        for s in range(2):
            close(t["pool"][int(kw["slots"][s])], pool[int(kw["slots"][s])])


def test_other_stream_and_two_at_once(cuda_device):
    """Two calls on two streams over slots of one pool."""
    mk = lambda i, P: batch(cuda_device, [90, 3, 40], 1, 2, 128, 128, "bf16", "softplus", True, seed=i,   # noqa: E731
                            slots=[3 * i, 3 * i + 1, 3 * i + 2], P=P)
    (a, ka), (b, kb) = mk(0, 6), mk(1, 6)
    b["pool"] = a["pool"]
    oa, pa = expect(a, ka)
    ob, pb = expect(b, kb)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, t, kw in ((streams[0], a, ka), (streams[1], b, kb)):
        with torch.cuda.stream(s):
            call(t, kw)
    torch.cuda.synchronize()
    close(a["o"], oa)
    close(b["o"], ob)
    close(a["pool"][:3], pa[:3])
    close(a["pool"][3:], pb[3:])


@pytest.mark.parametrize("per_head", [False, True])
def test_capture_and_replay(cuda_device, per_head):
    """A captured call replays over the rows, bounds and slots it finds then."""
    t, kw = batch(cuda_device, [40, 3, 1], 1, 2, 128, 128, "bf16", "softplus", per_head, P=8)
    call(t, kw)                                   # first use outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(t, kw)
    for seed, lens, slots in ((1, [1, 1, 1], [7, -1, 0]), (2, [2, 41, 1], [5, 6, 1]), (3, [0, 44, 0], [1, 2, 3])):
        u, ku = batch(cuda_device, lens, 1, 2, 128, 128, "bf16", "softplus", per_head, seed=seed, P=8, slots=slots,
                      behind=44 - sum(lens))
        for n in ("q", "k", "v", "g", "beta", "pool", "o"):
            t[n].copy_(u[n])
        kw["cu_seqlens"].copy_(ku["cu_seqlens"])
        kw["slots"].copy_(ku["slots"])
        o, pool = expect(t, kw)
        graph.replay()
        close(t["o"], o)
        close(t["pool"], pool)
    kda.kda_device_status()


def test_views_of_one_projection(cuda_device):
    """q, k, v, gate and beta as columns of one fused row, as a projection
    leaves them."""
    H, HV, D, T = 2, 4, 128, 100
    gen = torch.Generator().manual_seed(5)
    sizes = [H * D, H * D, HV * D, HV, HV]
    x = torch.randn(T, sum(sizes), generator=gen).to(torch.bfloat16).to(cuda_device)
    q, k, v, g, beta = x.split(sizes, 1)
    t, kw = batch(cuda_device, [60, 40], H, HV, D, D, "bf16", "softplus", True)
    t.update(q=q.unflatten(1, (H, D)), k=k.unflatten(1, (H, D)), v=v.unflatten(1, (HV, D)), g=g, beta=beta)
    check(t, kw)


def test_long_pool_offsets(cuda_device):
    """A slot whose state lies beyond 2^31 elements of the pool."""
    P, HV, D = 1030, 128, 128
    t, kw = batch(cuda_device, [2, 40], 1, HV, D, D, "bf16", "softplus", True, P=2, slots=[0, 1])
    small = t["pool"]
    t["pool"] = torch.empty(P, HV, D, D, device=cuda_device)
    assert (P - 1) * HV * D * D > 2 ** 31
    t["pool"][P - 2:] = small
    o, pool = expect(dict(t, pool=small), kw)
    kw["slots"] += P - 2
    call(t, kw)
    close(t["o"], o)
    close(t["pool"][P - 2:], pool)


def test_more_sequences_than_pages_in_one_decode_batch(cuda_device):
    """Hundreds of single rows beside a few long ones, lengths unknown to the host."""
    lens = [1] * 300 + [70, 40] + [2] * 100 + [90]
    check(*batch(cuda_device, lens, 1, 1, 128, 128, "bf16", "softplus", True))


# ------------------------------------------------------------- convolution
def conv_batch(dev, lens, C, K, dtype, seed=0, pad=0, slots=None, fresh=None, P=None, behind=0):
    gen = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    T, n = sum(lens) + behind, len(lens)
    P = P or n + 2
    slots = torch.randperm(P, generator=gen)[:n].tolist() if slots is None else slots
    t = {"x": torch.randn(T, C + pad, generator=gen).to(dt).to(dev)[:, :C],
         "w": torch.randn(C, K, generator=gen).to(dev) * 0.5, "bias": torch.randn(C, generator=gen).to(dev) * 0.1,
         "pool": torch.randn(P, K - 1, C, generator=gen).to(dt).to(dev),
         "y": torch.full((T, C), 0.0625, dtype=dt, device=dev)}
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev),
              slots=torch.tensor(slots, dtype=torch.int32, device=dev),
              fresh=None if fresh is None else torch.tensor(fresh, dtype=torch.uint8, device=dev))
    return t, kw


def conv_expect(t, kw, **more):
    host = lambda x: None if x is None else x.tolist()     # noqa: E731
    return packed.packed_conv(*(to_np(t[n]) for n in ("x", "w", "pool", "y", "bias")), cu=host(kw["cu_seqlens"]),
                              slots=host(kw["slots"]), fresh=host(kw["fresh"]), **more)


CONV = {
    "step": dict(lens=[1] * 11, C=256, K=4, dtype="bf16"),
    "short": dict(lens=[1, 2, 3, 0, 4, 1, 1, 2], C=128, K=4, dtype="f32", fresh=[0, 1, 0, 1, 0, 1, 0, 0]),
    "ragged": dict(lens=[700, 1, 33, 2900], C=640, K=4, dtype="bf16", fresh=[1, 0, 0, 1], behind=9, pad=8),
    "two_taps": dict(lens=[40, 5], C=128, K=2, dtype="bf16"),
    "three_taps": dict(lens=[2, 40, 5], C=384, K=3, dtype="f32", pad=4),
    "one_tap": dict(lens=[40, 5], C=128, K=1, dtype="f32"),
    "skipped": dict(lens=[4, 5, 6], C=128, K=4, dtype="bf16", slots=[2, -1, 0]),
}


@pytest.mark.parametrize("head_dim,silu", [(128, True), (0, True), (0, False)])
@pytest.mark.parametrize("name", CONV)
def test_convolution(cuda_device, name, head_dim, silu):
    t, kw = conv_batch(cuda_device, **CONV[name])
    y, pool = conv_expect(t, kw, head_dim=head_dim, silu=silu)
    kda.kda_packed_conv(t["x"], t["w"], t["pool"], t["bias"], y=t["y"], head_dim=head_dim, silu=silu, **kw)
    close(t["y"], y)
    assert np.array_equal(to_np(t["pool"]), pool)          # the windows are copies
    kda.kda_device_status()


def test_convolution_reports_bad_sequences(cuda_device):
    t, kw = conv_batch(cuda_device, [4, 5, 6, 3], 128, 4, "bf16", slots=[2, 2, 7, 1], P=6)
    y, pool = conv_expect(t, kw)
    kda.kda_packed_conv(t["x"], t["w"], t["pool"], t["bias"], y=t["y"], **kw)
    close(t["y"], y)
    assert np.array_equal(to_np(t["pool"]), pool)
    with pytest.raises(kda.KdaError):
        kda.kda_device_status()


def test_convolution_in_pieces_and_replayed(cuda_device):
    """A sequence run whole equals the same sequence a few rows at a time, the
    pieces of one row through a captured step."""
    C, T = 256, 23
    t, kw = conv_batch(cuda_device, [T], C, 4, "bf16", slots=[1], P=3)
    start = t["pool"].clone()
    whole = kda.kda_packed_conv(t["x"], t["w"], t["pool"], t["bias"], head_dim=128, **kw)
    end, pool = t["pool"].clone(), start.clone()
    slot = torch.tensor([1], dtype=torch.int32, device=cuda_device)
    x1, y1 = torch.empty(1, C, dtype=torch.bfloat16, device=cuda_device), None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1 = kda.kda_packed_conv(x1, t["w"], pool, t["bias"], head_dim=128, slots=slot)
    at, got = 0, []
    for n in (2, 1, 5, 1, 1, 3, 1, 9):
        piece = t["x"][at:at + n]
        if n == 1:
            x1.copy_(piece)
            graph.replay()
            got.append(y1.clone())
        else:
            got.append(kda.kda_packed_conv(piece, t["w"], pool, t["bias"], head_dim=128, slots=slot,
                                           cu_seqlens=torch.tensor([0, n], dtype=torch.int32, device=cuda_device)))
        at += n
    assert torch.equal(torch.cat(got), whole) and torch.equal(pool, end)


# ------------------------------------------------------------- together
@pytest.mark.parametrize("per_head", [False, True])
def test_layer_prefill_then_decode(cuda_device, per_head):
    """Convolutions, delta rule and group norm of one layer over a packed batch:
    the prompts whole, then token by token with the states the pools hold, equal
    the whole sequences at once."""
    dev, H, HV, D, dt = cuda_device, 2, 2, 128, torch.bfloat16
    gen = torch.Generator().manual_seed(9)
    full, prompt = [75, 40, 9], [70, 37, 4]
    T = sum(full)
    Cq, Cv = H * D, HV * D
    xs = torch.randn(T, 2 * Cq + Cv, generator=gen).to(dt).to(dev)
    g = torch.randn(T, HV, *(() if per_head else (D,)), generator=gen).to(dt).to(dev)
    beta, z = torch.randn(T, HV, generator=gen).to(dt).to(dev), torch.randn(T, Cv, generator=gen).to(dt).to(dev)
    w = (torch.randn(2 * Cq + Cv, 4, generator=gen) * 0.5).to(dev)
    gamma = (1 + 0.1 * torch.randn(Cv, generator=gen)).to(dev)
    A = torch.zeros(HV, device=dev)

    def layer(rows, cu, slots, pools, fresh):
        kw = dict(cu_seqlens=cu, slots=slots, fresh=fresh)
        x = xs[rows]
        q = kda.kda_packed_conv(x[:, :Cq], w[:Cq], pools[0], head_dim=128, **kw).unflatten(1, (H, D))
        k = kda.kda_packed_conv(x[:, Cq:2 * Cq], w[Cq:2 * Cq], pools[1], head_dim=128, **kw).unflatten(1, (H, D))
        v = kda.kda_packed_conv(x[:, 2 * Cq:], w[2 * Cq:], pools[2], **kw).unflatten(1, (HV, D))
        o = kda.kda_packed_fwd(q, k, v, g[rows], beta[rows], pools[3], A_log=A, gate_in_kernel="softplus",
                               g_per_head=per_head, scale=D ** -0.5, **kw)
        y, _, _ = kda.kda_group_norm_fwd(o.reshape(-1, 1, Cv), HV, gamma, None, z[rows][:, None], act="silu")
        return y[:, 0]

    def pools():
        junk = lambda *s: torch.full(s, float("nan"), device=dev)      # noqa: E731
        return [junk(5, 3, Cq).to(dt), junk(5, 3, Cq).to(dt), junk(5, 3, Cv).to(dt), junk(5, HV, D, D)]

    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)     # noqa: E731
    starts = [0, full[0], full[0] + full[1]]
    slots, fresh = i32([3, 0, 4]), torch.ones(3, dtype=torch.bool, device=dev)
    whole_pools = pools()
    whole = layer(slice(None), i32(starts + [T]), slots, whole_pools, fresh)
    part = pools()
    rows_p = [r for s, n in zip(starts, prompt) for r in range(s, s + n)]
    got = torch.empty_like(whole)
    got[rows_p] = layer(rows_p, i32([0, 70, 107, 111]), slots, part, fresh)
    for step in range(5):
        on = [i for i in range(3) if prompt[i] + step < full[i]]
        rows_d = [starts[i] + prompt[i] + step for i in range(3) if i in on]
        got[rows_d] = layer(rows_d, None, i32([[3, 0, 4][i] for i in on]), part, None)
    # both sides carry fp32 states and round q, k, v alike: what differs is the
    # order of sums, rounded once to bf16 in o and once in y
    ref = to_np(whole)
    assert np.all(np.abs(to_np(got) - ref) <= 2 ** -6 * np.abs(ref) + 2 ** -8 * np.abs(ref).max())
    for a, b in zip(part, whole_pools):
        live = [3, 0, 4]
        close(a[live].float(), to_np(b[live]))
    kda.kda_device_status()
