"""The drawing of tokens where few rows of a large vocabulary lie on the device: up
to 4 rows of 131072 tokens and more are cut over 16 CTAs each, more rows over 8.
And logits whose offsets pass 32 bits.  Tolerances are test_gpu_sample's."""
import numpy as np
import pytest
import torch

from test_gpu_sample import DT, _check, _draw, _logits
from weight_streaming_gemv_bf16_gb300 import binding as wb

pytestmark = pytest.mark.gpu

# the largest; top_k searched by one CTA, by all; borders of top_p and min_p; none
SETTINGS = [dict(temperature=0.0), dict(), dict(temperature=1.3, min_p=0.02), dict(top_p=0.9),
            dict(top_p=0.999, temperature=2.0), dict(top_k=50, top_p=0.95, temperature=0.8),
            dict(top_k=2500), dict(top_k=9000, top_p=0.97), dict(top_k=140000, top_p=0.5, min_p=0.001)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert wb.device_error(reset=True) == 0
    yield
    torch.cuda.synchronize()
    assert wb.device_error() == 0


@pytest.mark.parametrize("V,pad", [(151936, 0), (151936, 3), (131072, 0), (200001, 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 2, 4])
def test_few_rows_of_a_large_vocabulary(rows, dtype, V, pad):
    x, u = _logits(rows, V, dtype, seed=rows + pad, pad=pad, banned=0.01)
    for s in SETTINGS:
        _check(x, u, **s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_long_row_is_drawn_the_same_at_every_width(dtype):
    """1 and 4 rows in 16 CTAs each, 8 and 9 in 8 CTAs, 20 and 400 in fewer: the same token and
    probability, bit for bit."""
    x, u = _logits(20, 151936, dtype, seed=3)
    x, u = torch.cat([x] * 20), u * 20
    for s in SETTINGS:
        token, prob = _draw(x[:20], u[:20], **s)
        for n in (1, 4, 8, 9, 400):
            t, p = _draw(x[:n], u[:n], **s)
            assert np.array_equal(t, np.tile(token, 20)[:n]), (n, s)
            assert np.array_equal(p, np.tile(prob, 20)[:n]), (n, s)


@pytest.mark.parametrize("V", [131072, 151936])
def test_equals_across_all_slices(V):
    """Equal logits in every CTA's slice: the lowest indices are kept, the draw falls among them."""
    for dtype in DT:
        x = torch.full((4, V), 1.75, dtype=DT[dtype], device="cuda")
        us = [0.0, 0.5, 0.999, 1.0]
        for k in (0, 5, 70000):
            n = k or V
            token, prob = _draw(x, us, top_k=k)
            assert token.tolist() == [0, int(np.float32(0.5) * n), int(np.float64(np.float32(0.999)) * n), n - 1]
            assert np.allclose(prob, 1.0 / n, rtol=1e-7, atol=0)
        x[:, V - 3:] = 2.0
        token, prob = _draw(x, us, top_k=1)
        assert token.tolist() == [V - 3] * 4 and (prob == 1.0).all()


@pytest.mark.parametrize("at", [0, 9495, 9496, 75000, 151935])
def test_one_logit_that_rules_a_row_out(at):
    """A NaN or an infinity in any CTA's slice: no token, whatever is asked for."""
    for value in ("nan", "inf"):
        x, u = _logits(3, 151936, "f32", seed=5)
        x[1, at] = float(value)
        for s in SETTINGS:
            token, prob = _draw(x, u, **s)
            assert token[1] == -1 and np.isnan(prob[1]) and (token[[0, 2]] >= 0).all()


def test_logits_beyond_32_bits():
    """More than 2^31 logits: the last rows are drawn as they are alone."""
    V, rows = 151936, 14200
    some, u = _logits(8, V, "bf16", seed=6)
    x = some.repeat(rows // 8, 1)
    assert x.numel() > 1 << 31
    s = dict(temperature=0.9, top_p=0.95)
    token, prob = _draw(x, u * (rows // 8), **s)
    t, p = _draw(some, u, **s)
    assert np.array_equal(token, np.tile(t, rows // 8)) and np.array_equal(prob, np.tile(p, rows // 8))


@pytest.mark.parametrize("V", [700, 5000, 151936])
def test_zeros_of_both_signs_in_the_settings(V):
    x, u = _logits(2, V, "f32", seed=7)
    for s in (dict(top_p=0.0), dict(min_p=0.0), dict(temperature=0.0), dict(top_p=0.0, top_k=40)):
        token, prob = _draw(x, [0.0, 0.0], **s)
        other, q = _draw(x, [-0.0, -0.0], **{n: v if n == "top_k" else -0.0 for n, v in s.items()})
        assert np.array_equal(token, other) and np.array_equal(prob, q)
        assert (token >= 0).all()
