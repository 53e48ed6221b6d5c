"""Errors of the norms and of clipping name what was wrong."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cce():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tests.conftest import build_library
    build_library()
    import linear_cross_entropy_gb300
    return linear_cross_entropy_gb300


def test_names(cce):
    x, w = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")
    for call, words in [(lambda: cce.layer_norm(x, w, eps=-1.0), "cce_layer_norm_forward .eps"),
                        (lambda: cce.rms_norm(x, w, weight_offset=math.inf), "weight_offset finite"),
                        (lambda: cce.cce_clip_grads([w, w], 1.0), "given twice"),
                        (lambda: cce.cce_clip_grads([x, x[1:]], 1.0), "overlap"),
                        (lambda: cce.cce_clip_grads([w], 1.0, eps=-1.0), "eps")]:
        with pytest.raises(cce.CCEError, match=words) as e:
            call()
        assert e.value.status == 4
