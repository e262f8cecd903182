"""A layer of experts over a prompt on an MI355X takes a row of x for each token whose choices it is given, no more and no
fewer."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from rows_cases import cuda, weights  # noqa: E402


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import device

    torch.cuda.set_device(0)
    return device


@pytest.mark.parametrize("rows", [1, 7, 9, 16])
def test_rows_without_choices_or_choices_without_rows(dv, rows):
    rng = np.random.default_rng(rows)
    layer = dv.PromptExperts(*map(cuda, (*weights(rng, "mxfp4", 4, 256, 256), *weights(rng, "mxfp4", 4, 256, 128))))
    ids, probs = dv.route(torch.randn(8, 4, device="cuda", generator=torch.Generator("cuda").manual_seed(1)), 2)
    x = torch.randn(rows, 256, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
    with pytest.raises(ValueError, match="rows for the choices of 8 tokens"):
        layer(x, ids, probs)
    layer(x[:1].expand(8, 256).contiguous(), ids, probs)
