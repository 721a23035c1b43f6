"""A softmax scale of zero weighs all tokens alike, however large their scores; and other
scales at the ends of fp32's range."""
import pytest
import torch

from tests.test_gpu_paged_attention import Case, compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.0, -0.0])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("form,rows,G,D,window,sinks", [
    ("decode", (1, [700, 33]), 8, 128, 0, 0), ("varlen", (0, [(150, 100), (3, 200)]), 4, 64, 0, 0), ("decode", (2, [300]), 2, 256, 0, 0),
    ("varlen", (0, [(140, 300)]), 3, 128, 60, 5),
])
@pytest.mark.parametrize("large", [1.0, 2.0 ** 57])
def test_scale_of_zero(cuda_device, scale, fmt, form, rows, G, D, window, sinks, large):
    """Scores of 2^120 and more before the scale.  The oracle has the definition's 0 * score = 0."""
    case = Case(form, rows, 1, G, D, fmt, window, sinks, seed=300 + D, scale=scale)
    case.q = (case.q.float() * large).to(torch.bfloat16)
    if fmt == "bf16":
        case.c[0] = (case.c[0].float() * large).to(torch.bfloat16)
    else:
        case.s[0] *= large
    compare(case, case.run(cuda_device))
