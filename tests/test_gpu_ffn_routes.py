"""The feed-forward block's exact and 64-bit tests at the sizes that take the launches which
the sizes of test_gpu_ffn.py leave out: sums in parts of 256 x 256 tiles, 128 x 128 tiles of
rows with two slots, and every activation in the 256 x 256 tiles and their quarters."""
import pytest

import ffn_routes as routes
import test_gpu_ffn as whole

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("saved", [False, True], ids=["", "saved"])
@pytest.mark.parametrize("tokens,model,hidden,pad,off", routes.SHAPES)
def test_forward_exact(tokens, model, hidden, pad, off, saved):
    whole.test_forward_exact(tokens, model, hidden, pad, off, saved)


@pytest.mark.parametrize("tokens,model,hidden,pad,off", routes.SHAPES)
def test_backward_exact(tokens, model, hidden, pad, off):
    whole.test_backward_exact(tokens, model, hidden, pad, off)


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("tokens,model,hidden", routes.ACTIVATED)
def test_forward_and_checkpoint(tokens, model, hidden, act):
    whole.test_forward_and_checkpoint(tokens, model, hidden, act)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("tokens,model,hidden", routes.ACTIVATED)
def test_backward(tokens, model, hidden, act, fmt):
    whole.test_backward(tokens, model, hidden, act, fmt)
