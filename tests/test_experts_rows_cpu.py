"""What the binding looks at in the rows given to the experts, without a GPU: all four
tensors of an ExpertRows, since the kernels index each of them.  The tensors lie in host
memory and say that they are on the device; what passes the binding's checks would go on
to the library, which has no device here."""

from __future__ import annotations

import pytest
import torch

import combine_get_dispatch_05_amd as epm


class Placed(torch.Tensor):
    is_cuda = property(lambda self: True)
    place = 0

    def get_device(self):
        return self.place


def placed(t, at=0):
    t = t.as_subclass(Placed)
    t.place = at
    return t


def zeros(*shape, dtype=torch.int32):
    return placed(torch.zeros(shape, dtype=dtype))


GOOD = dict(expert_offsets=(5,), pair_row=(8,), pair_slot=(8,), row_pair=(4, 2))


def call(back, rows):
    buf, bf, f32 = epm.Buffer(2, 4), torch.bfloat16, torch.float32
    x, w13, w2 = zeros(4, 16, dtype=bf), zeros(4, 16, 16, dtype=bf), zeros(4, 16, 8, dtype=bf)
    if back:
        return buf.expert_ffn_backward(x, x, rows, zeros(4, 2, dtype=f32), w13, w2, zeros(8, 16, dtype=f32))
    return buf.expert_ffn(x, rows, zeros(4, 2, dtype=f32), w13, w2)


BAD = [(name, how) for name in GOOD for how in ("type", "dims", "stride", "place")]
BAD += [("expert_offsets", "length"), ("pair_slot", "length"), ("row_pair", "length")]


@pytest.mark.parametrize("back", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("name,how", BAD)
def test_rows_that_the_kernels_could_not_index(monkeypatch, name, how, back):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    shape = GOOD[name]
    bad = {"type": lambda: zeros(*shape, dtype=torch.int64),
           "dims": lambda: zeros(*shape, 1),
           "stride": lambda: placed(torch.zeros((*shape[:-1], 2 * shape[-1]), dtype=torch.int32)[..., ::2]),
           "place": lambda: placed(torch.zeros(shape, dtype=torch.int32), 1),
           "length": lambda: zeros(shape[0] - 1, *shape[1:])}[how]()
    rows = epm.ExpertRows(**{**{n: zeros(*s) for n, s in GOOD.items()}, name: bad})
    with pytest.raises((TypeError, ValueError)):
        call(back, rows)
