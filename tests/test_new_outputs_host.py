"""The new outputs of the 8-bit calls, on the CPU."""
import pytest
import torch

from newton_schulz_04_amd import _q8


@pytest.mark.parametrize("shapes", [[(3, 16)], [(3, 16), (4, 16)], [(3, 17), (4, 17), (0, 17)], [(3, 16), (4, 20)],
                                    [(0, 0), (2, 0)], [(5, 3), (7, 3)]])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_new_tensors_are_a_list(shapes, dtype):
    """A list, as the calls say, whether the tensors share a block or not: aligned to 16
    bytes, rows side by side, apart from one another."""
    got = _q8._empty(shapes, dtype, "cpu")
    assert type(got) is list and [tuple(t.shape) for t in got] == shapes
    for i, t in enumerate(got):
        assert t.dtype == dtype and t.is_contiguous() and (t.numel() == 0 or t.data_ptr() % 16 == 0)
        t.fill_(i)
    assert all(bool((t == i).all()) for i, t in enumerate(got))
