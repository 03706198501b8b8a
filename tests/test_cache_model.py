"""The plain model of the 4-bit cache against its definition (CPU)."""

import numpy as np
import pytest
import torch

import cache_model as M


def test_grids_are_the_formats():
    """The e4m3 grid is torch's float8_e4m3fn; the e2m1 grid is (1 + m/2) 2^(e-1), m/2 where e = 0."""
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(M.E4M3, t)
    e, m = np.arange(8) >> 1, np.arange(8) & 1
    np.testing.assert_array_equal(M.E2M1, np.where(e > 0, 2.0 ** (e - 1.0) * (1 + m / 2), m / 2))


def test_nearest_is_brute_force():
    rng = np.random.default_rng(1)
    x = np.concatenate([np.abs(rng.standard_normal(2000)) * 4, M.E2M1, (M.E2M1[1:] + M.E2M1[:-1]) / 2, [7, 1e9, np.inf]])
    got = M.nearest(x, M.E2M1)
    for v, i in zip(x, got):
        off = np.abs(np.minimum(v, 6.0) - M.E2M1)
        best = np.flatnonzero(off == off.min())
        assert i in best and (len(best) == 1 or i % 2 == 0), (v, i)
    s = torch.linspace(0, 448, 40001, dtype=torch.float64)
    want = s.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(M.nearest(s.float().double().numpy(), M.E4M3), want)


@pytest.mark.parametrize("exp", [0, -6, 5])
def test_held_values_are_bf16_and_near(exp):
    """Held values are bf16 values; each is within half the grid's widest step (2 of 6) of its scale
    and the scale's own rounding (2^-4 relative) of the original."""
    rng = np.random.default_rng(2)
    x = torch.tensor(rng.standard_normal((50, 64)) * 2.0 ** exp).bfloat16().double().numpy()
    c, s = M.quantise(x, exp)
    v = M.values(c, s, exp)
    np.testing.assert_array_equal(torch.tensor(v).bfloat16().double().numpy(), v)
    a = np.repeat(np.abs(x.reshape(50, -1, 16)).max(-1), 16, -1)
    assert (np.abs(v - x) <= a / 6 * (1 + 2.0 ** -4) + a * 2.0 ** -4).all()


def test_special_groups():
    x = np.zeros((5, 16))
    x[1, 3] = np.nan
    x[2, 5] = -np.inf
    x[3, :] = 5000.0
    x[4, 0] = -0.0
    x[4, 1] = 2.0 ** -12  # its scale rounds to 0
    c, s = M.quantise(x)
    assert s[0, 0] == 0 and not c[0].any()
    assert s[1, 0] == 127 and not c[1].any() and np.isnan(M.values(c, s)[1]).all()
    assert M.values(c, s)[2, 5] == -2688 and (M.values(c, s)[3] == 2688).all()
    assert s[4, 0] == 0 and not c[4].any()


def test_decode_of_the_model_is_plain_attention():
    """With every block taken, the model's decode is softmax attention over the held values."""
    rng = np.random.default_rng(3)
    m = M.Model(6, 2, 3, 2, 64, 128)
    assert m.reserve([300, 128])
    k, v = (rng.standard_normal((428, 2, 64)) for _ in "kv")
    hk, hv = m.append(k, v, [0, 300, 428], [0, 0])
    q = rng.standard_normal((2, 4, 64))
    out, lse, _, _, _ = m.decode(q, 0)
    for i, (a, b) in enumerate([(0, 300), (300, 428)]):
        kt, vt = (torch.tensor(t[a:b]).transpose(0, 1).repeat_interleave(2, 0) for t in (hk, hv))
        qt = torch.tensor(q[i])[:, None]
        want = torch.nn.functional.scaled_dot_product_attention(qt, kt, vt)[:, 0]
        np.testing.assert_allclose(out[i], want.numpy(), rtol=0, atol=1e-12)
        np.testing.assert_allclose(lse[:, i], torch.logsumexp(qt @ kt.transpose(1, 2) / 8, -1)[:, 0].numpy(), atol=1e-12)
