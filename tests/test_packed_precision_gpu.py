"""The chunk form of the packed delta rule keeps the accuracy of a recurrence in 32
bits: both against the FP64 oracle on the same inputs.

Tolerances.  The claim is a comparison, so the bound is the recurrence's own error:
a chunk rounds the state once where 64 tokens round it 64 times, and what its split
operands leave out is 2^-26 of a product.  On top, once: the state a chunk leaves
is a sum of rows that are each multiplied by a factor exp(G_C - G_j) from the
special-function unit (PTX ex2.approx: off by up to 2^-22 of its value), where the
recurrence multiplies expf's; a sum of rows that are each off by at most 2^-22 is off
by 2^-22 of the norm where they do not cancel.  With decays around e^-1 only the last
few tokens count, the recurrence's roundings do not add up, and that term is
the larger one.  Outputs: both sides round to bf16 at
the end; a value goes to the other neighbour where its error crosses a border, so
the shares of such values compare as the errors do (counts of rare events, three
standard deviations allowed)."""
import numpy as np
import pytest
import torch

from helpers import to_np
from test_packed_gpu import batch, call, expect

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("z_mean", [0.0, -4.0, -8.0])
def test_chunks_are_as_exact_as_the_recurrence(cuda_device, z_mean):
    kw_ = dict(lens=[2048, 700], H=1, HV=2, Dk=128, Dv=128, dtype="bf16", gate="softplus", per_head=True, seed=11,
               z_mean=z_mean, scale=128 ** -0.5)
    off, flips = {}, {}
    for algo in ("tc", "simt"):
        t, kw = batch(cuda_device, **kw_)
        o, pool = expect(t, kw)
        call(t, kw, algo=algo)
        slots = kw["slots"].tolist()
        off[algo] = np.array([np.linalg.norm(to_np(t["pool"][s]) - pool[s]) / np.linalg.norm(pool[s]) for s in slots])
        flips[algo] = int((t["o"].cpu() != torch.from_numpy(o).to(torch.bfloat16)).sum())
    print(z_mean, off, flips)
    assert np.all(off["tc"] <= off["simt"] + 2.0 ** -22)
    assert flips["tc"] <= flips["simt"] + 3 * flips["simt"] ** 0.5 + 3
