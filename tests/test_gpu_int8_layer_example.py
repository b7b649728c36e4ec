"""The example layers: the int8 operators as one layer against its torch form on the same route, the same
layer with its rows laid out by expert in between bit for bit, and a routed layer's gradients."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def _example(name):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", name + ".py")
    spec = importlib.util.spec_from_file_location(name, path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens", [1, 16, 70, 200])
def test_int8_layer(tokens):
    # h and out are bf16: 2^-8 for out's rounding; a rounding of h that goes the other way (where fp32
    # sums differ) is 2^-8 of a value, and a code of h that flips by it is 1/127 of its row's largest, in
    # one of F inputs: below 1 % of the largest output
    assert _example("int8_layer").main(["--tokens", str(tokens), "--hidden", "512", "--ffn", "256", "--experts", "16",
                                        "--top-k", "4"]) <= 2.0 ** -8 + 0.01


@pytest.mark.parametrize("tokens", [1, 9, 60, 400])
def test_int8_layer_through_sorted_rows(tokens):
    """In fp32 without a shared expert both ways take the same roundings: a row's products do not depend on
    the rows beside it, and the weighted sums run in slot order."""
    import torch
    layer = _example("int8_layer").Int8Layer(tokens, 384, 256, 12, 3, shared=False, dtype=torch.float32)
    x = torch.randn((tokens, 384), device="cuda")
    one, two = torch.empty_like(x), torch.empty_like(x)
    layer(x, one)
    layer.sorted_call(x, two)
    assert torch.equal(one, two)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_training_gradients(score):
    # fp32 on both sides: products of up to 256 terms and sums over up to 512 tokens, each off by at most
    # 512 * 2^-24 = 3e-5 of the sum of magnitudes, and by its square root on average
    assert _example("train_routed_layer").main(["--score", score]) <= 3e-5
