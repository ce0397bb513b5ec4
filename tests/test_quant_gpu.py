"""quantize_blocks on the GPU: every bit against its definition in fp32, and the values
against the fp64 ones.

An e4m3 number is off by at most half a step: 2^-4 of the value, or 2^-10 (half the
smallest step) times the scale; 448 / a', the product with it and scale each add one fp32
rounding (2^-24), which may also decide a tie the other way: within the same half step.
"""
import numpy as np
import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from oracle import moe as om
from tests.layers_parity import DT, f64, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from vocabulary_lm_cross_gb300 import build
    build.build()


def expected(x: torch.Tensor, down: int, across: int):
    """(bytes, scale) in fp32 on the CPU."""
    xf = x.cpu().float()
    R, C = xf.shape
    amax = torch.from_numpy(om.block_maxima(xf.numpy(), down, across)).float().clamp(min=2.0 ** -100)
    amax = torch.where(torch.isnan(amax), float("nan"), amax)

    def each(s):
        return s.repeat_interleave(down, 0).repeat_interleave(across, 1)[:R, :C]

    q = (xf * each(torch.tensor(448.0) / amax)).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), amax / 448.0


def check_values(q, scale, x, down, across):
    s = om.spread(f64(scale), down, across, q.shape)
    want = f64(x)
    bound = (2.0 ** -4 * np.abs(want) + 2.0 ** -10 * s) * (1 + 2.0 ** -20)
    assert (np.abs(f64(q.float()) * s - want) <= bound).all()


def raw(t):
    return t.view(torch.uint8).cpu()


SHAPES = [(1, 1), (1, 128), (128, 1), (3, 130), (64, 264), (129, 257), (200, 1000), (300, 640), (1, 4096),
          (1001, 136)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,C", SHAPES)
def test_rows_and_transposed(R, C, dtype):
    g = gen(R + C)
    x = randn(g, (R, C), DT[dtype], pad=(R * C) % 9)
    x[0, 0] *= 100
    both = v.quantize_blocks(x, transposed=True)
    q, s = expected(x, 1, 128)
    assert torch.equal(raw(both.q), q) and torch.equal(both.scale.cpu(), s)
    check_values(both.q, both.scale, x, 1, 128)
    qt, st = expected(x.t().contiguous(), 1, 128)
    assert both.qt.shape == (C, R) and both.qt.stride(0) % 16 == 0
    assert torch.equal(raw(both.qt), qt) and torch.equal(both.scale_t.cpu(), st)
    check_values(both.qt, both.scale_t, x.t(), 1, 128)
    one = v.quantize_blocks(x)
    assert one.qt is None and torch.equal(raw(one.q), q) and torch.equal(one.scale.cpu(), s)
    other = v.quantize_blocks(x, rows=False, transposed=True)
    assert other.q is None and torch.equal(raw(other.qt), qt) and torch.equal(other.scale_t.cpu(), st)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,C", SHAPES)
def test_square(R, C, dtype):
    x = randn(gen(R * C), (R, C), DT[dtype], sigma=0.02, pad=(R + C) % 9)
    r = v.quantize_blocks(x, square=True, transposed=True)
    q, s = expected(x, 128, 128)
    assert torch.equal(raw(r.q), q) and torch.equal(r.scale.cpu(), s)
    assert torch.equal(raw(r.qt), q.t()) and torch.equal(r.scale_t.cpu(), s.t())
    check_values(r.q, r.scale, x, 128, 128)


@pytest.mark.parametrize("R,C", [(5, 100), (256, 512), (130, 264)])
def test_a_batch_is_its_matrices(R, C):
    x = torch.randn((3, R + 2, C), generator=gen(5)).bfloat16().cuda()[:, 1:R + 1]
    for square in (False, True):
        r = v.quantize_blocks(x, square=square, transposed=True)
        for e in range(3):
            one = v.quantize_blocks(x[e], square=square, transposed=True)
            for a, b in zip(r, one):
                assert torch.equal(raw(a[e]), raw(b))


@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("R,C,dtype", [(3001, 4104, "bf16"), (8200, 4096, "f16"), (3001, 4104, "f32"),
                                       (3001, 4101, "bf16")])
def test_more_tiles_than_run_at_once(R, C, dtype, square):
    """The whole is its parts of 256 rows, which the tests above hold against the oracle."""
    x = randn(gen(C), (R, C), DT[dtype])
    x *= torch.exp2(torch.arange(R, device="cuda") % 7 - 3)[:, None].to(x.dtype)
    for rows, transposed in ((True, True), (True, False), (False, True)):
        r = v.quantize_blocks(x, square=square, rows=rows, transposed=transposed)
        for at in range(0, R, 256):
            part = v.quantize_blocks(x[at:at + 256], square=square, rows=rows, transposed=transposed)
            n, b = min(256, R - at), at // 128
            if rows:
                s = r.scale[b:b + part.scale.shape[0]] if square else r.scale[at:at + n]
                assert torch.equal(r.q[at:at + n].view(torch.uint8), part.q.view(torch.uint8))
                assert torch.equal(s, part.scale)
            if transposed:
                assert torch.equal(r.qt[:, at:at + n].view(torch.uint8), part.qt.view(torch.uint8))
                assert torch.equal(r.scale_t[:, b:b + part.scale_t.shape[1]], part.scale_t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zeros_tiny_values_infinities_and_nans(dtype):
    x = torch.zeros((130, 640), dtype=DT[dtype])
    x[1, 0:128] = 2.0 ** -120
    x[2, 128:256] = 2.0 ** -101
    x[3, 256:384] = 3e38
    x[4, 300] = float("inf")
    x[5, 400] = float("nan")
    x[6, 500], x[6, 511] = float("inf"), float("nan")
    x = x.cuda()
    r = v.quantize_blocks(x, transposed=True)
    val = r.q.float() * r.scale.repeat_interleave(128, 1)[:, :640]
    assert torch.isnan(val[4, 256:384]).all() and torch.isnan(val[5, 384:512]).all()
    assert torch.isnan(val[6, 384:512]).all()
    rest = torch.isnan(val)
    rest[4, 256:384] = rest[5, 384:512] = rest[6, 384:512] = False
    assert not rest.any()
    assert (val[0] == 0).all() and (r.scale[0] == np.float32(2.0 ** -100) / np.float32(448)).all()
    assert (val[3, 256:384] == x[3, 256:384].float()).all() or \
        ((val[3, 256:384] / x[3, 256:384].float() - 1).abs() < 1e-6).all()
    assert (val[1, :128] == 0).all()  # 448 2^-20 rounds to 0
    vt = r.qt.float() * r.scale_t.repeat_interleave(128, 1)[:, :130]
    assert torch.isnan(vt[300, :128]).all() and torch.isnan(vt[400, :128]).all()
    assert not torch.isnan(vt[300, 128:]).any() and not torch.isnan(vt[301]).any()
    sq = v.quantize_blocks(x, square=True)
    vs = sq.q.float() * sq.scale.repeat_interleave(128, 0)[:130].repeat_interleave(128, 1)
    assert torch.isnan(vs[:128, 256:512]).all() and not torch.isnan(vs[:, :256]).any()


@pytest.mark.parametrize("shape", [(256, 256), (130, 261)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_one_bad_value_spoils_its_block_only(dtype, shape):
    """Of either sign, beside larger patterns of the other, aligned rows or not."""
    x = randn(gen(7), shape, DT[dtype])
    spots = {(1, 3): float("inf"), (70, 130): float("-inf"), (129, 5): float("nan"), (128, 200): -float("nan")}
    for at, value in spots.items():
        x[at] = value
    clean = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    for square in (False, True):
        r, c = (v.quantize_blocks(t, square=square, transposed=True) for t in (x, clean))
        for q, s, qc, sc, flip in ((r.q, r.scale, c.q, c.scale, False), (r.qt, r.scale_t, c.qt, c.scale_t, True)):
            R, C = q.shape
            down = 128 if square else 1
            bad = torch.zeros((R, C), dtype=torch.bool, device="cuda")
            for i, j in spots:
                i, j = (j, i) if flip else (i, j)
                i0, j0 = i // down * down, j // 128 * 128
                bad[i0:i0 + down, j0:j0 + 128] = True
            val = q.float() * s.repeat_interleave(down, 0)[:R].repeat_interleave(128, 1)[:, :C]
            assert torch.equal(torch.isnan(val), bad)
            assert torch.equal(q.view(torch.uint8)[~bad], qc.view(torch.uint8)[~bad])


def test_empty_and_a_stream():
    r = v.quantize_blocks(torch.empty((0, 256), device="cuda"), transposed=True)
    assert r.q.shape == (0, 256) and r.qt.shape == (256, 0) and r.scale.shape == (0, 2)
    x = randn(gen(2), (256, 384), torch.bfloat16)
    want = v.quantize_blocks(x, transposed=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = v.quantize_blocks(x, transposed=True)
    s.synchronize()
    assert all(torch.equal(raw(a), raw(b)) for a, b in zip(got, want))


def test_rows_beyond_2_to_the_31_elements():
    C = 16384
    R = 2 ** 31 // C + 130
    x = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    tail = randn(gen(3), (130, C), torch.bfloat16)
    x[-130:] = tail
    r = v.quantize_blocks(x, transposed=True)
    assert torch.equal(raw(r.q[-130:]), raw(v.quantize_blocks(tail).q))
    first = R - 130
    assert first % 128 == 0
    t = v.quantize_blocks(tail, rows=False, transposed=True)
    assert torch.equal(raw(r.qt[:, first:]), raw(t.qt))
    assert torch.equal(r.scale_t[:, first // 128:], t.scale_t)
