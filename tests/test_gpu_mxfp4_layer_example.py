"""The example layer of the MXFP4 operators against its torch form on the same route: h and out are
bf16, so a value is off by one rounding (2^-8) where fp32 sums differ; a rounding of h that goes the
other way moves an E2M1 code of the down product by one step of at most a quarter of its block's
largest value in one of F inputs."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 16, 70, 200])
def test_example_layer(tokens):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_layer.py")
    spec = importlib.util.spec_from_file_location("mxfp4_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    # 2^-8 for out's rounding; h codes that flip are rare, each at most 1/4 of a value of about
    # 1/sqrt(F) of the output: 1 % of the largest output covers several
    assert m.main(["--tokens", str(tokens), "--hidden", "512", "--ffn", "256", "--experts", "16", "--top-k", "4"]) <= 2.0 ** -8 + 0.01
