"""Options of an optimiser's groups, without a GPU."""
import math

import pytest
import torch


@pytest.fixture(scope="module")
def cce():
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    return linear_cross_entropy_gb300


def params():
    return [torch.nn.Parameter(torch.zeros(4))]


@pytest.mark.parametrize("option", [dict(state_bits=16), dict(state_bits=4), dict(lr=-1.0), dict(lr=math.nan),
                                    dict(betas=(0.9, 1.0)), dict(betas=(-0.1, 0.9)), dict(eps=-1.0), dict(eps=math.nan),
                                    dict(weight_decay=-0.1)])
def test_a_groups_options_are_checked(cce, option):
    name = next(iter(option))
    with pytest.raises(ValueError, match=name):
        cce.AdamW([dict(params=params()), dict(params=params()) | option])
    opt = cce.AdamW(params())
    with pytest.raises(ValueError, match=name):
        opt.add_param_group(dict(params=params()) | option)
    assert len(opt.param_groups) == 1


def test_groups_keep_their_own(cce):
    opt = cce.AdamW([dict(params=params(), state_bits=8, lr=torch.tensor(0.1)), dict(params=params(), weight_decay=0.0)], lr=1e-2)
    assert [g["state_bits"] for g in opt.param_groups] == [8, 32] and opt.param_groups[1]["lr"] == 1e-2
    opt.add_param_group(dict(params=params(), betas=(0.0, 0.5)))
    assert opt.param_groups[2]["betas"] == (0.0, 0.5) and opt.param_groups[2]["eps"] == 1e-8
