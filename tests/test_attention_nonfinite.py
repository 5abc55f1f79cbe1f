"""Prompt attention where q, k or v hold infinities or NaN that a row sees: a logit of -inf gives its key no weight;
one of +inf or NaN, or only -inf ones, make the row NaN; an element of V that is not finite reaches every row that sees
it, whatever its weight: NaN for NaN or infinities of both signs, otherwise that infinity."""
import numpy as np
import pytest

from oracle import attention as ref
from tests.test_attention import DTYPES, _assert_within, _np, _prompt_tolerance, _rand, _starts, bl, torch  # noqa: F401

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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("more", [0, 300])
def test_a_first_tile_of_keys_without_weight(bl, dtype, d, more):  # noqa: F811
    """Every key of the first 64 (and 130) rows has the logit -inf: rows behind them are the rest's, rows among them NaN."""
    lens, hq, hkv = [90, 300] + [9] * more, 4, 2
    m, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (_rand((m, h, d), 91 + i, DTYPES[dtype]) for i, h in enumerate((hq, hkv, hkv)))
    q[..., 5] = -q[..., 5].abs() - 0.25
    k[:64, :, 5] = INF
    k[90:90 + 130, :, 5] = INF
    out = _np(bl.attention(q, k, v, _starts(lens))).reshape(m, hq, d)
    assert np.isnan(out[:64]).all() and np.isnan(out[90:220]).all()
    finite = k.clone()
    finite[:64, :, 5], finite[90:220, :, 5] = 0.0, 0.0
    want, spread, reach = np.zeros((m, hq, d)), np.zeros((m, hq, d)), np.zeros((m, hq, 1))
    for a, skip, b in [(0, 64, 90), (90, 130, 390)] + [(int(x), 0, int(y)) for x, y in zip(cu[2:-1], cu[3:])]:
        w = ref.attention(_np(q)[a + skip:b], _np(finite)[a + skip:b], _np(v)[a + skip:b], [0, b - a - skip], d ** -0.5)
        want[a + skip:b], spread[a + skip:b], reach[a + skip:b] = w
    rows = np.concatenate([np.arange(64, 90), np.arange(220, m)])
    _assert_within(out[rows], want[rows], _prompt_tolerance(want, spread, reach, max(lens), d, dtype)[rows])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [None, -0.2])
@pytest.mark.parametrize("more", [0, 300])
def test_keys_that_are_not_finite(bl, dtype, d, scale, more):  # noqa: F811
    """An infinity in a key is a logit of its sign times q's: -inf and the key has no weight, +inf and the row is NaN, as
    it is for 0 * inf, for infinities of both signs, and for NaN."""
    lens, hq, hkv = [40, 333, 120] + [9] * more, 6, 2
    m, group, sign = sum(lens), 3, -1.0 if scale else 1.0
    q, k, v = (_rand((m, h, d), 101 + i, DTYPES[dtype]) for i, h in enumerate((hq, hkv, hkv)))
    q[::3, :, 2] = 1.0                    # values without a second part
    q[::5, :, 2] = -1.0
    q[60, :, 2] = 0.0
    k[7, :, 2], k[41, :, 2], k[100, 0, 3], k[373 + 64, 1, d - 1] = INF, INF, -INF, INF
    k[200, 0, 4], k[200, 0, 5] = INF, -INF
    k[330, 1, 8] = NAN
    out = _np(bl.attention(q, k, v, _starts(lens), scale=scale)).reshape(m, hq, d)
    qn, kn, vn = _np(q).astype(np.float64), _np(k).astype(np.float64), _np(v)
    with np.errstate(invalid="ignore"):
        logits = sign * np.stack([_odd_products(qn[:, h], kn[:, h // group]) for h in range(hq)])
    bound = np.concatenate([[0], np.cumsum(lens)])
    finite = np.where(np.isfinite(kn), kn, 0.0)
    checked = {"nan": 0, "no weight": 0}
    use = d ** -0.5 if scale is None else scale
    for a, b in zip(bound[:3], bound[1:4]):
        seen = np.tril(np.ones((b - a, b - a), bool))
        for h in range(hq):
            odd = logits[h, a:b, a:b]
            nan_row = (seen & (np.isnan(odd) | (odd == INF))).any(1)
            none = seen & (odd == -INF)
            kk, vv = finite[a:b, h // group], vn[a:b, h // group]
            nan_row |= ~(seen & ~none).any(1)
            assert np.isnan(out[a:b, h][nan_row]).all(), (a, h)
            p = ref._softmax(use * (qn[a:b, h] @ kk.T), seen & ~none)
            reach = np.where(seen, abs(use) * (np.abs(qn[a:b, h]) @ np.abs(kk).T), 0).max(1)[:, None]
            ok = ~nan_row
            _assert_within(out[a:b, h][ok], (p @ vv)[ok], _prompt_tolerance(p @ vv, p @ np.abs(vv), reach, b - a, d, dtype)[ok], f"{a} {h}")
            checked["nan"] += int(nan_row.sum())
            checked["no weight"] += int((none.any(1) & ok).sum())
    assert checked["nan"] > 50 and checked["no weight"] > 50
    assert np.isfinite(out[bound[3]:]).all()


def _odd_products(q, k):
    """Sums of q_d k_d over the dims in which k is not finite (0 for keys that are), [rows][keys]."""
    out = np.zeros((q.shape[0], k.shape[0]))
    for j in np.flatnonzero(~np.isfinite(k).all(1)):
        dims = ~np.isfinite(k[j])
        out[:, j] = (q[:, dims] * k[j, dims]).sum(1)
    return out
