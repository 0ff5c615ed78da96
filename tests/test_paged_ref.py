"""The float64 statement of the paged cache's operators, against torch's own e4m3
rounding, against complex multiplication and against itself token by token."""

import numpy as np
import torch

from tests import paged_ref as R


def test_e4m3_table_and_rounding_match_torch():
    b = torch.arange(256, dtype=torch.uint8)
    t = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, R.E4M3, equal_nan=True)
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(4096, generator=g) * 60, torch.randn(4096, generator=g) * 0.01,
                   torch.tensor(sorted(set(R.E4M3[~np.isnan(R.E4M3)])))[:-1]
                   .float().add(torch.tensor(sorted(set(R.E4M3[~np.isnan(R.E4M3)])))[1:].float()) / 2])
    x = x.clamp(-448, 448)
    want = x.to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.round_e4m3(x.double().numpy()), want)
    assert np.isnan(R.round_e4m3([np.inf, -np.inf, np.nan])).all()


def test_least_scale():
    for amax in (0.0, 1e-40, 448.0, np.nextafter(448.0, 500), 447.9, 1.0, 1.75, 1.7500001, 3e38):
        s = R.least_scale(amax)
        assert amax <= 448 * s
        assert s == 2.0 ** -100 or amax > 448 * s / 2


def test_rotation_is_complex_multiplication():
    rng = np.random.default_rng(3)
    x = rng.standard_normal(128)
    f = 10000.0 ** (-np.arange(32) / 32)
    for inter in (False, True):
        y, _ = R.rotated(x, 777, f, inter)
        a = np.arange(0, 64, 2) if inter else np.arange(32)
        b = np.arange(1, 64, 2) if inter else np.arange(32, 64)
        z = (x[a] + 1j * x[b]) * np.exp(1j * 777 * f)
        assert np.allclose(y[a], z.real, atol=1e-12) and np.allclose(y[b], z.imag, atol=1e-12)
        assert np.array_equal(y[64:], x[64:])


def test_a_prompt_at_once_or_token_by_token_gives_one_cache():
    """With values whose magnitudes stay within e4m3's normal range of their page, the
    order in which the tokens come does not show."""
    rng = np.random.default_rng(5)
    n = 40
    x = torch.tensor(rng.choice([-1, 1], (n, 2, 128)) * rng.uniform(0.5, 2, (n, 2, 128))
                     * np.linspace(0.5, 6, n)[:, None, None]).bfloat16()
    v = x.flip(0)
    empty = lambda: (torch.zeros((3, 2, 16, 128), dtype=torch.uint8),) * 2 + \
        (torch.ones(3, 2),) * 2 + (torch.tensor([[2, 0, 1]]),)  # noqa: E731
    one, many = R.RefCache(*empty()), R.RefCache(*empty())
    one.append(x, v, [n], [0, n])
    for i in range(n):
        many.append(x[i:i + 1], v[i:i + 1], [i + 1])
    for w in range(2):
        assert np.array_equal(one.scale[w], many.scale[w])
        assert np.array_equal(one.val[w], many.val[w])


def test_rounding_again_as_a_scale_grows_stays_within_a_step():
    """Tokens one by one, each larger than those before, so that a page's scale grows again and
    again and earlier values sink among e4m3's subnormals, 2^-9 of the scale apart. A value is
    rounded once more at each growth, by at most 2^-10 of the scale it goes to; the scales at
    least double, so the sum is below 2^-9 of the last one (a first rounding while the value was
    normal, 2^-4 of a power of two below 2^-6 of the scale s at which it first is not, is below
    2^-11 s and does not change that). Rounding at once is off by at most 2^-10 of it, so the two
    are at most one subnormal step apart. Normal values are the same either way."""
    rng = np.random.default_rng(6)
    n = 16
    x = rng.standard_normal((n, 2, 128)) * np.exp2(np.linspace(-9, 9, n))[:, None, None] \
        * rng.choice([1, 2.0 ** -4, 2.0 ** -8], (n, 2, 128))
    x = torch.tensor(x).bfloat16()
    empty = lambda: (torch.zeros((1, 2, 16, 128), dtype=torch.uint8),) * 2 + \
        (torch.ones(1, 2),) * 2 + (torch.tensor([[0]]),)  # noqa: E731
    one, many = R.RefCache(*empty()), R.RefCache(*empty())
    one.append(x, x, [n], [0, n])
    for i in range(n):
        many.append(x[i:i + 1], x[i:i + 1], [i + 1])
    s = one.scale[0][0]
    assert np.array_equal(s, many.scale[0][0])
    exact = x.double().numpy().transpose(1, 0, 2) / s[:, None, None]
    a, b = one.val[0][0], many.val[0][0]
    small = (np.abs(a) <= 2.0 ** -6) & (np.abs(b) <= 2.0 ** -6)
    assert np.array_equal(a[~small], b[~small])
    assert (np.abs(b - exact)[small] < 2.0 ** -9).all() and (np.abs(a - b)[small] <= 2.0 ** -9).all()
    assert (a != b).any()
    # rounded at scale 1, then again at scale 4
    first = R.round_e4m3(0.058349609375)
    assert R.round_e4m3(first / 4) * 4 == 0.0625 and R.round_e4m3(0.058349609375 / 4) * 4 == 0.0546875
