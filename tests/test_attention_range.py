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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("more", [0, 300])
def test_scale_zero_of_large_products(bl, dtype, more):  # noqa: F811
    """scale 0 is the running mean, however large the products of q and k are."""
    lens, hq, hkv, d = [150, 70] + [9] * more, 6, 2, 64
    m, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (_rand((m, h, d), 131 + i, DTYPES[dtype]) for i, h in enumerate((hq, hkv, hkv)))
    out = bl.attention(q * 2.0 ** 62, k * 2.0 ** 62, v, _starts(lens), scale=0.0)  # products to 2^127
    want, spread, reach = ref.attention(_np(q), _np(k), _np(v), cu, 0.0)
    _assert_within(_np(out).reshape(m, hq, d), want, _prompt_tolerance(want, spread, reach, max(lens), d, dtype))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [10, 19, 26, 36])
@pytest.mark.parametrize("more", [0, 300])
def test_large_channels_of_a_row_fp32(bl, d, power, more):  # noqa: F811
    """One channel of q, of k or of v 2^power times the others, fp32: an element is held to 2^-39 of its row's largest
    (q and k: that times the other factor's sum in the logit), a weight to 2^-36 of the largest p_ij max |v_j|."""
    lens, hq, hkv = [150, 70] + [9] * more, 6, 2
    m, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)])
    for which in range(3):
        t = [_rand((m, h, d), 141 + i, torch.float32) for i, h in enumerate((hq, hkv, hkv))]
        t[which][..., 11] *= 2.0 ** power
        if which < 2:  # the channel itself adds little to the logits, so that the others' rounding counts
            t[1 - which][..., 11] *= 2.0 ** -power
        q, k, v = t
        out = _np(bl.attention(q, k, v, _starts(lens))).reshape(m, hq, d)
        qn, kn, vn = (_np(x).astype(np.float64) for x in t)
        want, spread, reach = ref.attention(qn, kn, vn, cu, d ** -0.5)
        per_head = lambda x: x.repeat(hq // hkv, 1)  # noqa: E731
        top = lambda x: np.abs(x).max(-1, keepdims=True)  # noqa: E731
        # the largest of any row of the sequence stands for that of the rows seen
        seq = np.repeat(np.arange(len(lens)), lens)
        largest = lambda x: np.stack([x[seq == s].max(0) for s in range(len(lens))])[seq]  # noqa: E731
        held = d ** -0.5 * 2.0 ** -39 * (top(qn) * largest(per_head(np.abs(kn).sum(-1, keepdims=True)))
                                         + np.abs(qn).sum(-1, keepdims=True) * largest(per_head(top(kn))))
        tol = _prompt_tolerance(want, spread, reach, max(lens), d, "f32") + 2 * held * spread
        tol = tol + 2.0 ** -39 * largest(per_head(top(vn)))
        tol = tol + 2.0 ** -36 * np.array(lens)[seq][:, None, None] * largest(per_head(top(vn))) * largest(per_head(np.abs(vn) / top(vn)))
        _assert_within(out, want, tol, f"{which}")
