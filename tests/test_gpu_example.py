"""The hybrid stack of examples/: its parts run together and agree with each other."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "hybrid_stack.py")


@pytest.fixture(scope="module")
def stack():
    spec = importlib.util.spec_from_file_location("hybrid_stack", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    from gated_delta_rule_07_gb300 import build
    build.build()
    return module


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
def test_steps_agree_with_drafted_tokens(stack, dtype):
    """The same tokens one at a time and all at once.  The ways differ in their roundings: bf16
    activations of four layers (2^-8 each, a few roundings a layer), and cache pages whose scale
    grew in steps (codes rounded twice: up to 2^-7 of a page's largest value for int8, 2^-4 of
    each value for e4m3, averaged over the keys).  A wrong state, page or position makes them
    differ by their size."""
    steps, drafted = stack.serve(steps=12, dtype=dtype)
    assert torch.isfinite(steps.float()).all()
    off = (steps.float() - drafted.float()).norm() / drafted.float().norm()
    assert off < 0.06, float(off)


def test_prompt_in_pieces(stack):
    """A prompt in one call and in three: pages are continued inside a call's rows."""
    gen = torch.Generator("cuda").manual_seed(9)
    lens = [150, 41]
    x = torch.randn(2, 160, stack.HIDDEN, device="cuda", generator=gen).bfloat16()

    def run(cuts):
        s, at, out = stack.Stack(2), [0, 0], None
        for cut in cuts:
            rows = torch.cat([x[n, at[n]:at[n] + cut[n]] for n in range(2)])
            out = s.extend(rows, cut)
            at = [a + c for a, c in zip(at, cut)]
        assert s.held.tolist() == lens
        return torch.stack([out[cuts[-1][0] - 1], out[-1]]).float()

    a, b = run([lens]), run([[100, 1], [17, 30], [33, 10]])
    assert (a - b).norm() / a.norm() < 0.06


def test_norm_weights_are_tuned(stack):
    losses = stack.tune()
    assert losses[-1] < 0.02 * losses[0]
