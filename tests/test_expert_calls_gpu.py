"""Calls of the experts' operators that their documentation allows, and results that have to
follow from others'."""
import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from examples import expert_mlp as ex

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


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


@pytest.mark.parametrize("R", [100, 128, 300])
def test_dweight_of_experts_that_all_start_at_the_end(R):
    a, sa = torch.ones((40, 304), device="cuda").to(FP8)[:, :R], torch.ones((40, -(-R // 128)), device="cuda")
    off = torch.full((4,), R, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = v.block_linear_dweight(a, sa, a, sa, offsets=off, dev_err=err)
    assert int(err) == 0 and got.shape == (3, 40, 40) and not got.any()
    keep = torch.ones((3, 40, 40), device="cuda")
    v.block_linear_dweight(a, sa, a, sa, offsets=off, dev_err=err, dweight=keep, accumulate=True)
    assert int(err) == 0 and (keep == 1).all()


def test_a_plan_of_no_experts_is_refused():
    with pytest.raises(v.capi.VlmceError):
        v.describe_block_linear_plan(16, 128, 128, 0)
    assert v.describe_block_linear_plan(16, 128, 128, 1).kernel == "small"
