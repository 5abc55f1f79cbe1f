"""Prompt attention at the ends of fp32's range, and with channels of very different sizes in a row, against the
definition in 64 bits within the bounds that include/bitlinear.h states."""
import numpy as np
import pytest

from oracle import attention as ref
from tests.test_attention import DTYPES, _assert_within, _np, _prompt_tolerance, _rand, _starts, bl, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [-95, -60, 60, 95, 110, 120])
@pytest.mark.parametrize("more", [0, 300])
def test_large_keys_and_small_queries(bl, dtype, d, power, more):  # noqa: F811
    """K times 2^power and q times 2^-power have the logits that they had (powers of two are exact). q's elements
    stay above fp32's smallest normal number, or are 0."""
    lens, hq, hkv = [150, 70] + [9] * more, 6, 2
    m, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (_rand((m, h, d), 111 + i, DTYPES[dtype]) for i, h in enumerate((hq, hkv, hkv)))
    q, k = (torch.where(x.abs() < 0.05, torch.zeros_like(x), x) for x in (q, k))  # 2^-120 * 0.05 > 2^-126
    out = bl.attention(q * 2.0 ** -power, k * 2.0 ** power, v, _starts(lens))
    want, spread, reach = ref.attention(_np(q), _np(k), _np(v), cu, d ** -0.5)
    _assert_within(_np(out).reshape(m, hq, d), want, _prompt_tolerance(want, spread, reach, max(lens), d, dtype))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [-122, -110, -90, 110])
@pytest.mark.parametrize("more", [0, 300])
def test_small_and_large_values_fp32(bl, d, power, more):  # noqa: F811
    """V times 2^power, fp32: besides the terms of the other tests an element of v is held to 2^-137 (and a result to
    fp32's smallest step, 2^-149)."""
    lens, hq, hkv = [150, 70] + [9] * more, 6, 2
    m, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (_rand((m, h, d), 121 + i, torch.float32) for i, h in enumerate((hq, hkv, hkv)))
    v = v * 2.0 ** power
    out = _np(bl.attention(q, k, v, _starts(lens))).reshape(m, hq, d).astype(np.float64)
    want, spread, reach = ref.attention(_np(q), _np(k), _np(v), cu, d ** -0.5)
    tol = _prompt_tolerance(want, spread, reach, max(lens), d, "f32") - 1e-30 + 2.0 ** -137 + 2.0 ** -149
    _assert_within(out, want, tol)
