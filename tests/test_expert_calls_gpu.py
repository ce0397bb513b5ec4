"""Calls of the experts' operators that their documentation allows, and results that have to
follow from others'."""
import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from examples import expert_mlp as ex

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from vocabulary_lm_cross_gb300 import build
    build.build()


def test_the_example_serves_with_the_weights_that_it_has_trained():
    sizes = dict(E=5, H=136, n=200, k=2)
    _, few, _ = ex.main(T=150, **sizes)
    m = ex.Experts(**sizes)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((150, sizes["H"]), generator=g, device="cuda").bfloat16()
    experts, weights = m.route(x)
    _, grads = ex.train_step(m, x, experts, weights, torch.ones_like(x))
    before = ex.serve(m, x[:4].clone(), experts[:4], weights[:4])
    for name in m.master:
        m.master[name].add_(grads[name], alpha=-1e-3)
    m.sync()
    after = ex.serve(m, x[:4].clone(), experts[:4], weights[:4])
    assert not torch.equal(before, after)
    assert torch.equal(few, after)
