"""The outputs that the packed bindings allocate."""
import torch

from gated_delta_rule_157_b200 import _lib


def test_rows_that_may_be_left_out_start_as_zeros(monkeypatch):
    monkeypatch.setattr(torch, "empty", lambda shape, **kw: torch.full(shape, float("nan"), **kw))
    cu, slots = torch.tensor([0, 2], dtype=torch.int32), torch.tensor([-1], dtype=torch.int32)
    for c, s in ((cu, None), (None, slots), (cu, slots)):
        assert (_lib._packed_out((3, 2), torch.float32, "cpu", c, s) == 0).all()
    assert _lib._packed_out((3, 2), torch.bfloat16, "cpu", None, None).dtype == torch.bfloat16      # every row is written
