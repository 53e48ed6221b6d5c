"""States loaded into parameters of other strides, without a GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def cce():
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    return linear_cross_entropy_gb300


def saved(opt, **state):
    return {"state": {0: {"step": 3} | state}, "param_groups": opt.state_dict()["param_groups"]}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_states_take_the_parameters_strides(cce, dtype):
    p = torch.nn.Parameter(torch.zeros(6, 8).to(dtype).t())
    opt = cce.AdamW([p])
    m, v, w = (torch.randn(8, 6) for _ in range(3))
    opt.load_state_dict(saved(opt, exp_avg=m, exp_avg_sq=v, master=w))
    for k, t in (("exp_avg", m), ("exp_avg_sq", v), ("master", w)):
        own = opt.state[p][k]
        assert torch.equal(own, t) and own.stride() == p.stride() and own.dtype == torch.float32 and not own.requires_grad
        assert own.data_ptr() != t.data_ptr()
    assert opt.state[p]["step"] == 3


def test_the_same_strides_are_copied(cce):
    p = torch.nn.Parameter(torch.zeros(8, 6))
    opt = cce.AdamW([p])
    m = torch.randn(8, 6)
    opt.load_state_dict(saved(opt, exp_avg=m, exp_avg_sq=m))
    m.zero_()
    assert opt.state[p]["exp_avg"].all() and opt.state[p]["exp_avg"].data_ptr() != opt.state[p]["exp_avg_sq"].data_ptr()


def test_8_bit_states_keep_theirs(cce):
    p = torch.nn.Parameter(torch.zeros(6, 8).t())
    opt = cce.AdamW([p], state_bits=8, min_8bit_size=1)
    codes = torch.arange(48, dtype=torch.uint8).view(8, 6).view(torch.float8_e4m3fn)
    opt.load_state_dict(saved(opt, exp_avg=codes, exp_avg_rms=codes, exp_avg_scale=torch.ones(1), rms_scale=torch.ones(1)))
    own = opt.state[p]["exp_avg"]
    assert own.dtype == codes.dtype and own.stride() == codes.stride()  # which a step refuses
    assert torch.equal(own.view(torch.uint8), codes.view(torch.uint8))
