"""Prompt attention where q, k or v hold infinities or NaN that a row sees: an element of V that is not finite reaches
every row that sees it, whatever its weight: NaN for NaN or infinities of both signs, otherwise that infinity."""
import numpy as np
import pytest

from tests.test_attention import DTYPES, _rand, _starts, bl, torch  # noqa: F401

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def _kind(x):
    """0 finite, 1 +inf, 2 -inf, 3 NaN."""
    return torch.where(torch.isnan(x), 3, torch.where(x == INF, 1, torch.where(x == -INF, 2, 0)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("more", [0, 300])
@pytest.mark.parametrize("steep", [False, True])
def test_values_that_are_not_finite_keep_their_kind(bl, dtype, d, more, steep):  # noqa: F811
    """Infinities and NaN of V in the first, masked tile of a prompt, in tiles that later rows see whole, and before
    keys whose logits are 200 powers of two larger (every weight before them is 0 in fp32): each row that sees them
    has their kind in that dim and finite values elsewhere, whether a tile's keys are split over two waves or
    (with 300 sequences more) not."""
    lens, hq, hkv = [40, 700, 1, 130] + [9] * more, 4, 2
    m, starts = sum(lens), np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (_rand((m, h, d), 71 + i, DTYPES[dtype]) for i, h in enumerate((hq, hkv, hkv)))
    if steep:
        q[..., 0] = 8.0
        k[..., 0] = 0.0
        for row in (39, 140, 300, 739, 800):  # scale * 8 * k = 140 > 200 ln 2
            k[row, :, 0] = 140.0 / (8.0 * d ** -0.5)
    bad = [(0, 3, INF), (20, 4, -INF), (39, 5, INF), (5, 6, NAN), (7, 9, INF), (30, 9, -INF), (12, 10, INF), (13, 10, INF),
           (40, 0, INF), (43, 1, -INF), (104, 2, NAN), (200, 3, -INF), (201, 11, INF), (600, 11, -INF), (739, d - 1, -INF),
           (740, 8, INF), (741 + 60, 33, -INF), (741 + 70, 34, INF), (741 + 129, 35, NAN), (741, 36, INF)]
    want = torch.zeros((m, hkv, d), dtype=torch.int64, device="cuda")
    for row, dim, value in bad:
        v[row, :, dim] = value
        end = int(starts[np.searchsorted(starts, row, side="right")])
        code = 3 if value != value else 1 if value > 0 else 2
        seen = want[row:end, :, dim]
        want[row:end, :, dim] = torch.where((seen == 0) | (seen == code), code, 3)
    out = bl.attention(q, k, v, _starts(lens)).view(m, hq, d)
    got, expected = _kind(out.float()), want.repeat_interleave(hq // hkv, 1)
    wrong = (got != expected).nonzero()
    assert len(wrong) == 0, (len(wrong), wrong[0].tolist(), int(got[tuple(wrong[0])]), int(expected[tuple(wrong[0])]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("more", [0, 300])
def test_no_value_reaches_a_row_without_weights(bl, dtype, more):  # noqa: F811
    """A row whose logits are NaN, or all -inf, is NaN in every dim, also where V holds an infinity."""
    lens, hq, hkv, d = [100] + [9] * more, 4, 2, 64
    m = sum(lens)
    q, k, v = (_rand((m, h, d), 81 + i, DTYPES[dtype]) for i, h in enumerate((hq, hkv, hkv)))
    v[2, :, 7] = INF
    q[50, 1, 3] = NAN          # a row of NaN logits
    q[70, :, 5] = INF          # logits of both infinities
    k[0, 1, 9], q[0, 2:, 9] = INF, -2.0  # the first row sees one key, of logit -inf
    out = bl.attention(q, k, v, _starts(lens)).view(m, hq, d)
    assert torch.isnan(out[50, 1]).all() and torch.isnan(out[70]).all() and torch.isnan(out[0, 2:]).all()
    assert (out[50, 0, 7] == INF).all() and torch.isfinite(out[1, :2]).all()
