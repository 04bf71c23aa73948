"""The binding's reading of rows without a GPU: views of two and three dimensions, columns of wider rows, give the pointer and
stride that the general rule (leading dimensions of more than one entry nest) gives, and what does not nest is refused."""
import itertools

import pytest
import torch

import selective_state_space_14_amd as ssd
from tests.test_binding_streams import OnGpu


def general(t):
    """The rule for any number of dimensions; None where the rows are not a uniform number of elements apart."""
    rs, step = None, 1
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if rs is None:
            rs = st
        elif st != rs * step:
            return None
        step *= n
    return rs


@pytest.mark.parametrize("shape", [(1, 8), (5, 8), (5, 1), (1, 1, 8), (1, 6, 8), (5, 1, 8), (5, 6, 8), (2, 3, 4, 8)])
def test_columns_of_wider_rows(shape):
    for lead, pad in itertools.product((0, 3), (0, 4)):
        wide = torch.zeros(shape[:-1] + (lead + shape[-1] + pad,)).as_subclass(OnGpu)
        t = wide[..., lead:lead + shape[-1]]
        p, rs = ssd._Call(t, "t").rows(t, "t", torch.float32, t.shape)
        assert p == t.data_ptr()
        if any(n > 1 for n in shape[:-1]):
            assert rs == general(t)
        else:
            assert rs >= shape[-1]


def test_rows_that_do_not_nest():
    wide = torch.zeros(5, 7, 8).as_subclass(OnGpu)
    for t in (wide[:, :6], wide.transpose(0, 1), wide[..., ::2], wide[::2], torch.zeros(8, 5).as_subclass(OnGpu).t()):
        want = general(t) if t.stride(-1) == 1 else None
        c = ssd._Call(t, "t")
        if want is None:
            with pytest.raises(ValueError, match="t: "):
                c.rows(t, "t", torch.float32, t.shape)
        else:
            assert c.rows(t, "t", torch.float32, t.shape) == (t.data_ptr(), want)
    t = wide[:, :6]
    for shape, T, err in (((5, 6, 7), torch.float32, ValueError), ((5, 6, 8), torch.bfloat16, TypeError)):
        with pytest.raises(err, match="t: expected"):
            ssd._Call(t, "t").rows(t, "t", T, torch.Size(shape))
