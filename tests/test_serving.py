"""The rotation of queries and keys, attention behind a shared prefix, the bounds of cached blocks, the choice by them and
attention over chosen blocks, on the GPU against the oracle's 64-bit definitions.

Tolerances, per element, u = 2^-24. Rotation: cos and sin are off by at most u of 1 after their rounding, their product
with the magnitude and an element's with them by u each, the difference by u of itself: 4 u magnitude (|a| + |b|) + u |y|
covers the four roundings of either term. A norm's sum of d squares is off by (d + 1) u of itself at most, so its root
by half of that; the mean, eps, the root, the division and two products round once each: (d / 2 + 7) u of the element.
Attention: as in test_attention.py; behind a prefix the fp32 sum of d products is off by (d + 2) u reach, q in two fp16
parts by 2^-22 reach, the weights by 2^-11 (bf16: fp16, u = 2^-11) or 2^-22 of themselves, or 2^-39 of their block's
largest (counted as 2^-38 grain)."""
import numpy as np
import pytest

from oracle import attention as cached_ref
from oracle import serving as ref
from tests.test_attention import DTYPES, _assert_within, _i32, _np, _Paged, _rand, _starts, bl, torch  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0**-24


def _cu(cu):
    return None if cu is None else cu.cpu().numpy()


# ---------------------------------------------------------------- rotation

def _check_rotate(bl, lens, begin, hq, hkv, d, rot, dtype, interleaved=False, norm=(True, True), magnitude=1.0, eps=1e-5, packed=True,
                  freq=None, sd=1.0, out="new", outside=(0, 0)):
    m = sum(lens) + sum(outside)
    qkv = _rand((m, (hq + 2 * hkv) * d), 13 * m + hq + rot, DTYPES[dtype], sd)
    q, k, _ = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    was = _np(q), _np(k)
    freq = bl.rotary_frequencies(rot, 10000.0) if freq is None else freq
    gains = [1 + 0.3 * _rand((d,), 5 + i, torch.float32) if n else None for i, n in enumerate(norm)]
    cu = _starts(lens) + outside[0] if packed else None
    where = {"new": None, "in place": (q, k), "given": tuple(torch.full_like(x.contiguous(), 7.0) for x in (q, k))}[out]
    got = bl.rotate(q, k, freq, _i32(begin), cu, interleaved=interleaved, q_gain=gains[0], k_gain=gains[1], eps=eps, magnitude=magnitude, out=where)
    at = ref.positions(begin, None if cu is None else cu.cpu().numpy(), m)
    used = at >= 0
    for x, y, gain in zip(was, got, gains):
        assert y.dtype == DTYPES[dtype] and y.shape == x.shape
        want, size = ref.rotate(x[used], at[used], freq.cpu().numpy(), interleaved, None if gain is None else _np(gain), np.float32(eps),
                                np.float32(magnitude))
        rel = (4 if gain is None else 4 + d / 2 + 7) * U
        tol = rel * size * max(1.0, abs(magnitude)) + U * np.abs(want) + 1e-37
        if dtype == "bf16":
            tol = tol + 2.0**-8 * np.abs(want)
        _assert_within(_np(y)[used], want, tol, f"{lens} {begin}")
        if out != "new":
            np.testing.assert_array_equal(_np(y)[~used], x[~used] if out == "in place" else 7.0)
    if out == "in place":
        assert got[0].data_ptr() == q.data_ptr()
        np.testing.assert_array_equal(_np(qkv)[:, (hq + hkv) * d:], _np(_rand((m, (hq + 2 * hkv) * d), 13 * m + hq + rot, DTYPES[dtype], sd))[:, (hq + hkv) * d:])
    return got


ROTATIONS = [  # lens, begin, q heads, kv heads, d, rotary dim
    ([1], [0], 20, 5, 128, 128), ([1], [1023], 1, 1, 64, 16), ([3, 0, 70], [9, 5, 131072], 7, 1, 128, 64), ([5, 2], [0, 77], 4, 4, 64, 64),
    ([130], [3], 32, 8, 128, 32), ([1] * 70, list(range(0, 7000, 100)), 6, 2, 64, 32), ([300, 1, 200], [0, 2**20, 4], 12, 4, 128, 112),
    ([0, 0, 17], [1, 1, 2], 40, 2, 64, 48), ([600], [10], 33, 11, 128, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [(True, True), (False, False)])
@pytest.mark.parametrize("lens,begin,hq,hkv,d,rot", ROTATIONS)
def test_rotate_against_the_definition(bl, lens, begin, hq, hkv, d, rot, norm, interleaved, dtype):  # noqa: F811
    _check_rotate(bl, lens, begin, hq, hkv, d, rot, dtype, interleaved, norm)
    if all(n == 1 for n in lens):
        _check_rotate(bl, lens, begin, hq, hkv, d, rot, dtype, interleaved, norm, packed=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["in place", "given"])
def test_rotate_rows_that_are_left(bl, out, dtype):  # noqa: F811
    """Unused slots and rows before and behind the sequences; in place on slices of the projection's rows, of which V stays."""
    _check_rotate(bl, [4, 3, 90], [10, -1, 0], 8, 2, 128, 64, dtype, out=out, outside=(2, 5))
    _check_rotate(bl, [1, 1, 1], [10, -1, 0], 8, 2, 64, 64, dtype, out=out, packed=False, interleaved=True)


@pytest.mark.parametrize("norm", [(True, False), (False, True)])
def test_rotate_norm_of_one_side(bl, norm):  # noqa: F811
    _check_rotate(bl, [33, 4], [0, 900], 6, 2, 128, 128, "f32", norm=norm)


def test_rotate_far_positions(bl):  # noqa: F811
    """Angles of the last positions that there are, and of frequencies above 1: no digit of the angle is lost."""
    _check_rotate(bl, [1, 1, 3], [2**31 - 1, 2**31 - 2, 2**31 - 2], 4, 1, 128, 128, "f32", norm=(False, False))
    _check_rotate(bl, [1, 40], [2**24 + 1, 12345678], 4, 1, 64, 64, "f32", freq=torch.linspace(-3.0, 9.7, 32, device="cuda"), norm=(False, False))


@pytest.mark.parametrize("magnitude,eps,sd", [(1.37, 1e-6, 1.0), (-0.5, 0.0, 1.0), (0.0, 1e-5, 1.0), (1.0, 1e-5, 1e-4), (1.0, 0.1, 1e3)])
def test_rotate_magnitudes(bl, magnitude, eps, sd):  # noqa: F811
    _check_rotate(bl, [50], [7], 8, 2, 64, 32, "f32", magnitude=magnitude, eps=eps, sd=sd)


def test_rotate_scaled_frequencies(bl):  # noqa: F811
    for kw in ({"scaling": "positions"}, {"scaling": "base"}, {"scaling": "parts", "length": 4096}):
        _check_rotate(bl, [9, 40], [30000, 0], 8, 2, 128, 128, "bf16", freq=bl.rotary_frequencies(128, 500000.0, factor=8.0, **kw))


def test_rotate_values_that_are_not_finite_stay_in_their_head(bl):  # noqa: F811
    q, k = _rand((3, 4, 64), 1, torch.float32), _rand((3, 2, 64), 2, torch.float32)
    f, at, cu, gain = bl.rotary_frequencies(32), _i32([5]), _starts([3]), torch.ones(64, device="cuda")
    clean = bl.rotate(q, k, f, at, cu, q_gain=gain, k_gain=gain)
    q[1, 2, 50], k[2, 0, 3] = float("nan"), float("inf")
    dirty = bl.rotate(q, k, f, at, cu, q_gain=gain, k_gain=gain)
    bad = [torch.zeros(x.shape[:2], dtype=torch.bool, device="cuda") for x in (q, k)]
    bad[0][1, 2] = bad[1][2, 0] = True
    for c, y, b in zip(clean, dirty, bad):
        assert torch.equal(c[~b], y[~b]) and not torch.isfinite(y[b]).all()
    assert torch.isnan(dirty[0][1, 2]).all()
    q[0, 0, 7] = 3e20  # its square passes fp32's range: the head's factor is 0
    huge = bl.rotate(q, k, f, at, cu, q_gain=gain, k_gain=gain)
    assert (huge[0][0, 0] == 0).all() and torch.equal(huge[0][0, 1:], clean[0][0, 1:])
    zero = bl.rotate(torch.zeros_like(q), torch.zeros_like(k), f, at, cu, q_gain=gain, k_gain=gain)
    assert (zero[0] == 0).all() and (zero[1] == 0).all()


@pytest.mark.parametrize("seqs", [64, 65, 4097, 9000])
def test_rotate_many_sequences(bl, seqs):  # noqa: F811
    """Every row finds its sequence among many, empty ones between them."""
    lens = [(i * 7) % 3 for i in range(seqs)]
    begin = [(i * 13) % 5000 for i in range(seqs)]
    _check_rotate(bl, lens, begin, 1, 1, 64, 16, "f32", norm=(False, False))


@pytest.mark.parametrize("cu", [[0, 300, 0, 300, 0], [300, 0, 300], [-4, 2**31 - 1, 5], [0] + [300, 0] * 40])
def test_offsets_out_of_order_stay_in_bounds(bl, cu):  # noqa: F811
    """Offsets that the rule for bad values covers: nothing outside the rows, the cache and the tables is touched."""
    seqs, hkv, d = len(cu) - 1, 2, 64
    c = _Paged(bl, [100] * seqs, [300] * seqs, hkv, d, 6)
    q, k = (torch.full((302, h, d), 3.0, device="cuda") for h in (8, hkv))
    table, lens, starts = _i32(c.table), _i32([100] * seqs), _i32(cu)
    guards = [torch.full((302, 8, d), 5.0, device="cuda"), torch.full((302, hkv, d), 5.0, device="cuda")]
    bl.rotate(q[1:301], k[1:301], bl.rotary_frequencies(64), lens, starts, out=(guards[0][1:301], guards[1][1:301]))
    bounds = bl.bounds_alloc(c.cache)
    bl.cache_bounds(c.cache, bounds, table, lens, starts, 300)
    sel = torch.full((302, hkv, 3), 5, dtype=torch.int32, device="cuda")
    bl.block_select(q[1:301], bounds, c.cache.k_scale, table, lens, 3, starts, out=sel[1:301])
    outs = [torch.full((302, 8 * d), 5.0, device="cuda") for _ in range(2)]
    bl.attention_selected(q[1:301], c.cache, table, lens, sel[1:301], starts, out=outs[0][1:301])
    bl.attention_shared(q[1:301], c.cache, table[0], lens[:1].contiguous(), table, lens, starts, out=outs[1][1:301])
    torch.cuda.synchronize()
    for g in (*guards, sel, *outs):
        assert (g[0] == 5).all() and (g[301] == 5).all() and torch.isfinite(g).all()


# ---------------------------------------------------------------- a shared prefix

def _tolerance(want, spread, reach, grain, blocks, d, dtype, behind):
    r = (32 + (d + 8 if behind else 0)) * U * reach + (blocks + 96 + (64 if behind else 0)) * U
    tol = 2 * r * spread + 2.0**-22 * grain + U * np.abs(want) + 1e-30
    if behind:
        tol = tol + 1.01 * (2.0**-11 if dtype == "bf16" else 2.0**-22) * spread
    if dtype == "bf16":
        tol = tol + 2.0**-8 * np.abs(want)
    return tol


def _check_shared(bl, c, prefix, length, lens, new, hq, dtype, seed=5, packed=True, scale=None, q=None, workspace=None):
    m, d = sum(new), c.d
    q = _rand((m, hq, d), seed, DTYPES[dtype], 1.5) if q is None else q
    cu = _starts(new) if packed else None
    guard = torch.full((m, hq * d), 7.0, dtype=DTYPES[dtype], device="cuda")
    out = bl.attention_shared(q, c.cache, _i32(prefix), _i32([length]), _i32(c.table), _i32(lens), cu, out=guard, scale=scale, workspace=workspace)
    want, spread, reach, grain = ref.attention_shared(_np(q), c.kc, c.ks, c.vc, c.vs, prefix, length, c.table, lens, _cu(cu),
                                                      d ** -0.5 if scale is None else scale)
    for s, (a, b) in enumerate(cached_ref._rows(_cu(cu), m, len(lens))):
        if lens[s] < 0:
            want[a:b] = 7
    _assert_within(_np(out).reshape(m, hq, d), want, _tolerance(want, spread, reach, grain, c.wide + len(prefix), d, dtype, True),
                   f"{length} {lens} {new}")
    return q, out


SHARED = [  # prefix length, lens, new, q heads, kv heads, d
    (1, [0], [1], 4, 1, 128), (64, [5, 0], [1, 1], 20, 5, 128), (65, [63, 64, 1], [1] * 3, 8, 8, 64), (1000, [3, 200, 0, 17], [1] * 4, 16, 2, 128),
    (63, [10], [40], 7, 1, 64), (700, [10, -1, 90], [2, 3, 5], 6, 2, 64), (130, [40 + i for i in range(70)], [1] * 70, 4, 2, 64),
    (2100, [9, 30], [4, 4], 12, 4, 128), (500, [300] * 9, [1] * 9, 40, 2, 64), (200, [0], [1], 64, 1, 128), (1300, [4000], [1], 4, 2, 128),
    (320, [(37 * i) % 100 for i in range(150)], [1 + i % 2 for i in range(150)], 4, 4, 64), (9000, [1, 2], [1, 1], 8, 1, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("length,lens,new,hq,hkv,d", SHARED)
def test_shared_against_the_definition(bl, length, lens, new, hq, hkv, d, dtype):  # noqa: F811
    blocks = -(-length // 64)
    c = _Paged(bl, lens + [length], new + [0], hkv, d, 21, wide=max(blocks, *(-(-(max(a, 0) + b) // 64) for a, b in zip(lens, new))))
    prefix, c.table = c.table[-1, :blocks], c.table[:-1]
    _check_shared(bl, c, prefix, length, lens, new, hq, dtype)
    if all(n == 1 for n in new):
        _check_shared(bl, c, prefix, length, lens, new, hq, dtype, packed=False)


def _behind(bl, length=200, lens=(70, 3), new=(2, 3), hkv=2, d=64, seed=4):  # noqa: F811
    c = _Paged(bl, list(lens) + [length], list(new) + [0], hkv, d, seed)
    prefix, c.table = c.table[-1].copy(), c.table[:-1].copy()
    return c, prefix


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("length", [-3, 0, 1, 64, 100, 10**6, 2**31 - 1])
def test_shared_lengths(bl, length, dtype):  # noqa: F811
    """No prefix, a part of what the table names, and more than it does."""
    c, prefix = _behind(bl)
    _check_shared(bl, c, prefix, length, [70, 3], [2, 3], 8, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_shared_scales(bl, scale, dtype):  # noqa: F811
    c, prefix = _behind(bl)
    _check_shared(bl, c, prefix, 190, [70, 3], [2, 3], 8, dtype, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_blocks_without_a_page(bl, dtype):  # noqa: F811
    """In the prefix, in the sequences, in both: rows that see nothing give 0; page 0 may hold anything."""
    c, prefix = _behind(bl)
    for t in (c.cache.k_scale, c.cache.v_scale):
        t[0] = float("nan")
    c.ks[0] = c.vs[0] = np.nan
    c.table[c.table == 0], prefix[prefix == 0] = 1, 1
    holes = prefix.copy()
    holes[1] = -1
    holes[2] = c.pages
    _check_shared(bl, c, holes, 200, [70, 3], [2, 3], 8, dtype)
    c.table[1] = -5
    _check_shared(bl, c, holes, 200, [70, 3], [2, 3], 8, dtype)
    none = np.full_like(prefix, -1)
    _, out = _check_shared(bl, c, none, 200, [70, 3], [2, 3], 8, dtype)
    assert (out[2:] == 0).all() and (out[:2] != 0).any()
    _, out = _check_shared(bl, c, none, 0, [70, 3], [2, 3], 8, dtype)
    assert (out[2:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_rows_that_are_not_finite(bl, dtype):  # noqa: F811
    c, prefix = _behind(bl)
    q, clean = _check_shared(bl, c, prefix, 200, [70, 3], [2, 3], 8, dtype)
    q = q.clone()
    q[1, 2, 5], q[4, 7, 63], q[0, 0, 0] = float("nan"), float("inf"), -float("inf")
    out = bl.attention_shared(q, c.cache, _i32(prefix), _i32([200]), _i32(c.table), _i32([70, 3]), _starts([2, 3])).view(5, 8, 64)
    bad = torch.zeros(5, 8, dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[4, 7] = bad[0, 0] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean.view(5, 8, 64)[~bad])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-25, 1e-6, 40.0, 1e12])
def test_shared_sizes_of_values(bl, size, dtype):  # noqa: F811
    """Queries of very different sizes beside scales that undo them, values whose scale differs by page: the weights of a
    page count beside the others' whatever its V is."""
    c, prefix = _behind(bl, length=400)
    for ours, theirs in ((c.ks, c.cache.k_scale), (c.vs, c.cache.v_scale)):
        ours *= np.float32(1 / size) if theirs is c.cache.k_scale else (10.0 ** np.linspace(-12, 12, c.pages)).astype(np.float32)[:, None]
        theirs.copy_(torch.tensor(ours))
    q = (_rand((5, 8, 64), 3, torch.float32) * size).to(DTYPES[dtype])
    _check_shared(bl, c, prefix, 400, [70, 3], [2, 3], 8, dtype, q=q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_channels_of_different_size(bl, dtype):  # noqa: F811
    """One channel of q 2^9 times the others, which K's codes make small there."""
    c, prefix = _behind(bl, length=300, d=128)
    c.kc[..., 5] = np.sign(c.kc[..., 5])
    c.cache.k.copy_(torch.tensor(cached_ref.stored(c.kc, c.place[0])))
    q = _rand((5, 4, 128), 3, torch.float32)
    q[..., 5] *= 512
    _check_shared(bl, c, prefix, 300, [70, 3], [2, 3], 4, dtype, q=q.to(DTYPES[dtype]))


def test_shared_peaks_page_by_page(bl):  # noqa: F811
    """Logits that rise from page to page by hundreds and fall again: the reference moves, the last page's weight counts."""
    c, prefix = _behind(bl, length=640)
    for order in (1, -1):
        c.ks[prefix[::order]] = (2.0 ** np.arange(len(prefix)))[:, None].astype(np.float32)[:, [0, 0]]
        c.cache.k_scale.copy_(torch.tensor(c.ks))
        _check_shared(bl, c, prefix, 640, [70, 3], [2, 3], 8, "f32")
        _check_shared(bl, c, prefix, 640, [70, 3], [2, 3], 8, "f32", scale=-0.2)


def test_shared_logits_past_the_integers_of_fp32(bl):  # noqa: F811
    """Logits of 2^30: one key takes all, and nothing turns into NaN."""
    c, prefix = _behind(bl, length=640)
    c.ks[:] = 2.0**26
    c.cache.k_scale.copy_(torch.tensor(c.ks))
    q = _rand((5, 8, 64), 3, torch.float32)
    out = bl.attention_shared(q, c.cache, _i32(prefix), _i32([640]), _i32(c.table), _i32([70, 3]), _starts([2, 3]))
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_stale_codes_behind_the_prefix(bl, dtype):  # noqa: F811
    c, prefix = _behind(bl)
    args = (_i32(prefix), _i32([131]), _i32(c.table), _i32([70, 3]), _starts([2, 3]))
    q = _rand((5, 8, 64), 3, DTYPES[dtype])
    before = bl.attention_shared(q, c.cache, *args)
    for codes, place in ((c.cache.k, c.place[0]), (c.cache.v, c.place[1])):
        codes[int(prefix[2])][:, torch.tensor(place[3:].ravel(), device="cuda")] = -128
    assert torch.equal(before, bl.attention_shared(q, c.cache, *args))


def test_shared_prefix_of_a_sequence_itself(bl):  # noqa: F811
    """A sequence split into a prefix of whole blocks and the rest: what attention over all of it gives."""
    c = _Paged(bl, [900], [1], 2, 128, 8)
    q = _rand((1, 8, 128), 3, torch.float32)
    whole = bl.attention_cached(q, c.cache, _i32(c.table), _i32([900]))
    for n in (1, 7, 14):
        got = bl.attention_shared(q, c.cache, _i32(c.table[0, :n]), _i32([64 * n]), _i32(c.table[:, n:]), _i32([900 - 64 * n]))
        np.testing.assert_allclose(_np(got), _np(whole), rtol=2e-5, atol=2e-5 * float(whole.abs().max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_outlier_channels_of_the_cache(bl, dtype):  # noqa: F811
    """Channels that set a page's scale beside others whose codes are small: what the others hold counts."""
    c, prefix = _behind(bl, length=500, d=128)
    for codes, ours, place in ((c.cache.k, c.kc, c.place[0]), (c.cache.v, c.vc, c.place[1])):
        ours[:] = np.clip(ours // 16, -7, 7)
        ours[..., 3], ours[..., 77] = 127, -120
        codes.copy_(torch.tensor(cached_ref.stored(ours, place)))
    _check_shared(bl, c, prefix, 500, [70, 3], [2, 3], 8, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_many_rows_and_pages(bl, dtype):  # noqa: F811
    """So many rows that a workgroup has the whole prefix and a wave more than 64 of its pages: every row as in a batch of
    a few, whose prefix is split (each within its own tolerance of the definition, u = 2^-24 or 2^-8)."""
    c, _ = _behind(bl, length=640, lens=(70,), new=(1,), hkv=1, d=64)
    prefix = _i32(np.random.default_rng(3).integers(0, c.pages, 300))
    few = _rand((3, 32, 64), 5, DTYPES[dtype], 1.5)
    n = 270
    out = [bl.attention_shared(few[torch.arange(m, device="cuda") % 3].contiguous(), c.cache, prefix, _i32([300 * 64 - 5]),
                               _i32(c.table).expand(m, -1).contiguous(), _i32([70] * m)) for m in (n, 3)]
    for i in range(3):
        assert (out[0][i::3] == out[0][i]).all()
    off = (out[0][:3].float() - out[1].float()).abs().max() / out[1].float().abs().max()
    assert off < (2.0**-7 if dtype == "bf16" else 2e-5)


# ---------------------------------------------------------------- bounds

@pytest.mark.parametrize("hkv,d", [(5, 128), (1, 64), (3, 128)])
@pytest.mark.parametrize("lens,new", [([0], [1]), ([63], [1]), ([64], [1]), ([5, 0, 130], [3, 64, 1]), ([17, 70, 128, 0], [1] * 4), ([0, 60], [200, 0]),
                                      ([1, 127], [63, 66]), ([100, -1, 3], [20, 4, 7]), ([60, 0] * 40, [9, 1] * 40)])
def test_bounds_against_the_definition(bl, lens, new, hkv, d):  # noqa: F811
    c = _Paged(bl, lens, new, hkv, d, 31)
    c.kc[::3, :, :, 0], c.kc[::2, :, :, 1], c.kc[:, :, :, 2] = -127, 127, 0
    c.kc[1::2, :, 5, 3] = -128  # what only an outsider's code can be
    c.cache.k.copy_(torch.tensor(cached_ref.stored(c.kc, c.place[0])))
    for cu in [_starts(new)] + ([None] if set(new) == {1} else []):
        bounds = bl.bounds_alloc(c.cache)
        bounds.fill_(9)
        bl.cache_bounds(c.cache, bounds, _i32(c.table), _i32(lens), cu, sum(new))
        want = np.full(bounds.shape, 9, np.int8)
        ref.cache_bounds(c.kc, want, c.table, lens, _cu(cu), sum(new))
        np.testing.assert_array_equal(bounds.cpu().numpy(), want)


@pytest.mark.parametrize("table,lens", [([[-1, 1]], [60]), ([[0, 99]], [60]), ([[0, -7]], [64]), ([[0, 1]], [126]), ([[0, 1]], [128]), ([[0, 1]], [2**31 - 3])])
def test_bounds_blocks_without_a_page(bl, table, lens):  # noqa: F811
    c = _Paged(bl, [0], [128], 2, 64, 12)
    bounds = bl.bounds_alloc(c.cache)
    want = np.zeros(bounds.shape, np.int8)
    bl.cache_bounds(c.cache, bounds, _i32(table), _i32(lens), _starts([5]), 5)
    ref.cache_bounds(c.kc, want, np.array(table), lens, [0, 5], 5)
    np.testing.assert_array_equal(bounds.cpu().numpy(), want)


# ---------------------------------------------------------------- selection

class _Bounds:
    def __init__(self, bl, lens, new, hkv, d, seed, wide=None, pages=None):  # noqa: F811
        rng = np.random.default_rng(seed)
        blocks = [-(-(max(a, 0) + b) // 64) for a, b in zip(lens, new)]
        self.wide = wide or max(1, max(blocks))
        self.pages = pages or sum(blocks) + 2
        self.table = rng.integers(0, self.pages, (len(lens), self.wide)) if pages else np.full((len(lens), self.wide), -1, np.int64)
        if not pages:
            order = rng.permutation(self.pages)
            for s, n in enumerate(blocks):
                self.table[s, :min(n, self.wide)] = order[sum(blocks[:s]):sum(blocks[:s]) + min(n, self.wide)]
        ends = np.sort(rng.integers(-127, 128, (self.pages, hkv, 2, d)), 2)[:, :, ::-1]
        self.bounds, self.ks = np.ascontiguousarray(ends).astype(np.int8), (0.5 + 2 * rng.random((self.pages, hkv))).astype(np.float32)

    def check(self, bl, q, lens, keep, cu, first, recent):  # noqa: F811
        m, hkv = q.shape[0], self.bounds.shape[1]
        out = torch.full((m, hkv, keep), 77, dtype=torch.int32, device="cuda")
        got = bl.block_select(q, torch.tensor(self.bounds).cuda(), torch.tensor(self.ks).cuda(), _i32(self.table), _i32(lens), keep, cu, first=first,
                              recent=recent, out=out)
        want = ref.block_select(_np(q), self.bounds, self.ks, self.table, lens, keep, _cu(cu), first, recent, 77)
        np.testing.assert_array_equal(got.cpu().numpy(), want)
        return got


SELECTS = [  # lens, new, q heads, kv heads, d, keep, first, recent
    ([0], [1], 4, 1, 128, 1, 0, 1), ([640], [1], 20, 5, 128, 4, 1, 2), ([63, 64, 65, 3000], [1] * 4, 8, 8, 64, 3, 0, 1), ([5000, 100], [1, 1], 7, 1, 64, 20, 2, 3),
    ([700, -1, 90, 4000], [2, 3, 5, 1], 6, 2, 64, 5, 1, 1), ([20000], [1], 128, 1, 128, 100, 0, 1), ([63] * 3, [4, 0, 2], 16, 2, 128, 1, 0, 1),
    ([37000], [3], 12, 4, 64, 570, 1, 2), ([40000], [1], 256, 2, 64, 8, 0, 8), ([9000] * 70, [1] * 70, 4, 2, 64, 17, 1, 1), ([640], [1], 4, 4, 128, 200, 1, 2),
    ([130000], [1], 8, 2, 128, 64, 1, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,new,hq,hkv,d,keep,first,recent", SELECTS)
def test_select_against_the_definition(bl, lens, new, hq, hkv, d, keep, first, recent, dtype):  # noqa: F811
    c = _Bounds(bl, lens, new, hkv, d, 3)
    q = _rand((sum(new), hq, d), 8, DTYPES[dtype], 1.5)
    c.check(bl, q, lens, keep, _starts(new), first, recent)
    if all(n == 1 for n in new):
        c.check(bl, q, lens, keep, None, first, recent)


@pytest.mark.parametrize("wide", [8192, 8193, 20000])
def test_select_wide_tables(bl, wide):  # noqa: F811
    """Tables of more blocks than keys fit LDS, full and nearly empty, and a length beyond the table."""
    for lens in ([wide * 64 - 1, 100], [600, wide * 64 + 5000]):
        c = _Bounds(bl, lens, [1, 1], 2, 64, 3, wide=wide, pages=300)
        c.check(bl, _rand((2, 4, 64), 8, torch.float32), lens, 33, None, 1, 2)


def test_select_ties_go_to_the_lower_block(bl):  # noqa: F811
    lens = [64 * 600 + 9]
    for pages in (1, 2, 5):
        c = _Bounds(bl, lens, [1], 2, 64, 3, pages=pages)
        for keep in (2, 7, 300, 600, 601, 900):
            c.check(bl, _rand((1, 4, 64), 8, torch.bfloat16), lens, keep, None, 0, 2)
    c.check(bl, torch.zeros((1, 4, 64), device="cuda"), lens, 7, None, 1, 2)  # every score 0


def test_select_scores_of_both_signs_and_no_pages(bl):  # noqa: F811
    lens = [64 * 300]
    c = _Bounds(bl, lens, [1], 1, 128, 3)
    c.bounds[::2] = -np.abs(c.bounds[::2])  # all keys negative
    c.bounds[..., 0, :] = np.maximum(c.bounds[..., 0, :], c.bounds[..., 1, :])
    q = _rand((1, 4, 128), 8, torch.float32).abs()
    c.check(bl, q, lens, 200, None, 0, 1)
    c.table[0, ::3] = -1
    c.table[0, 1::7] = c.pages + 3
    for keep in (20, 150, 250):
        c.check(bl, q, lens, keep, None, 1, 1)
    c.ks[3::5], c.ks[4::11] = np.nan, np.inf
    c.check(bl, q, lens, 90, None, 1, 1)


def test_select_queries_that_are_not_finite(bl):  # noqa: F811
    lens = [64 * 100, 64 * 90]
    c = _Bounds(bl, lens, [1, 1], 2, 64, 3)
    q = _rand((2, 8, 64), 8, torch.float32)
    q[0, 1, 5], q[1, 3, 7], q[1, 6, 9] = float("nan"), float("inf"), -float("inf")
    c.check(bl, q, lens, 9, None, 0, 1)
    c.check(bl, q * 1e-38, lens, 9, None, 0, 1)


# ---------------------------------------------------------------- attention over chosen blocks

def _check_selected(bl, c, lens, new, hq, sel, dtype, packed=True, scale=None, seed=5, workspace=None):  # noqa: F811
    m, d = sum(new), c.d
    q = _rand((m, hq, d), seed, DTYPES[dtype], 1.5)
    cu = _starts(new) if packed else None
    guard = torch.full((m, hq * d), 7.0, dtype=DTYPES[dtype], device="cuda")
    out = bl.attention_selected(q, c.cache, _i32(c.table), _i32(lens), _i32(sel), cu, out=guard, scale=scale, workspace=workspace)
    want, spread, reach, grain = ref.attention_selected(_np(q), c.kc, c.ks, c.vc, c.vs, c.table, lens, sel, _cu(cu), d ** -0.5 if scale is None else scale)
    for s, (a, b) in enumerate(cached_ref._rows(_cu(cu), m, len(lens))):
        if lens[s] < 0:
            want[a:b] = 7
    _assert_within(_np(out).reshape(m, hq, d), want, _tolerance(want, spread, reach, grain, sel.shape[2], d, dtype, False), f"{lens} {new}")
    return q, out


SELECTED = [  # lens, new, q heads, kv heads, d, keep
    ([0], [1], 4, 1, 128, 1), ([1000], [1], 20, 5, 128, 9), ([63, 64, 65, 3], [1] * 4, 8, 8, 64, 2), ([5000, 100], [1, 1], 7, 1, 64, 60),
    ([700, -1, 90], [2, 3, 5], 6, 2, 64, 5), ([400], [30], 40, 2, 64, 4), ([9000], [1], 32, 8, 128, 64), ([1500] * 70, [1] * 70, 16, 2, 128, 12),
    ([5000], [1], 64, 1, 128, 70), ([(41 * i) % 900 for i in range(150)], [1 + i % 2 for i in range(150)], 12, 4, 64, 7), ([20000], [1], 4, 1, 64, 300),
    ([3000], [5], 24, 3, 128, 40),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,new,hq,hkv,d,keep", SELECTED)
def test_selected_against_the_definition(bl, lens, new, hq, hkv, d, keep, dtype):  # noqa: F811
    """Lists with holes, entries beyond the table and behind the row, and blocks listed more than once, in no order."""
    c = _Paged(bl, lens, new, hkv, d, 77)
    rng = np.random.default_rng(keep)
    sel = rng.integers(-1, c.wide, (sum(new), hkv, keep))
    sel[rng.random(sel.shape) < 0.05] = c.wide + 3
    sel[0, 0, 0] = 0
    _check_selected(bl, c, lens, new, hq, sel, dtype)
    if all(n == 1 for n in new):
        _check_selected(bl, c, lens, new, hq, sel, dtype, packed=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_selected_rows_that_see_nothing(bl, dtype):  # noqa: F811
    c = _Paged(bl, [300, 40], [2, 1], 2, 64, 4)
    for t in (c.cache.k_scale, c.cache.v_scale):
        t[0] = float("nan")
    c.ks[0] = c.vs[0] = np.nan
    c.table[c.table == 0] = -1
    sel = np.array([[[-1, -1, -2**31], [4, 0, 1]], [[2**31 - 1, 9, -1], [2, 3, -1]], [[1, 2, 3], [0, 0, 0]]])
    _, out = _check_selected(bl, c, [300, 40], [2, 1], 8, sel, dtype)
    out = out.view(3, 2, 4, 64)
    assert (out[0, 0] == 0).all() and (out[1, 0] == 0).all() and (out[2, 0] == 0).all()


def test_selected_all_blocks_is_attention_over_the_cache(bl):  # noqa: F811
    c = _Paged(bl, [700, 333], [1, 1], 2, 128, 8)
    q = _rand((2, 8, 128), 3, torch.float32)
    sel = torch.arange(c.wide, dtype=torch.int32, device="cuda").expand(2, 2, c.wide).contiguous()
    assert torch.equal(bl.attention_selected(q, c.cache, _i32(c.table), _i32([700, 333]), sel),
                       bl.attention_cached(q, c.cache, _i32(c.table), _i32([700, 333])))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_selected_long_lists_of_many_rows(bl, dtype):  # noqa: F811
    """So many rows that one workgroup has a whole list and a wave more than 64 of its blocks, and some whose lists are
    split, both read past the caches: every row as in a batch of a few."""
    c = _Paged(bl, [1200], [1], 2, 64, 8)
    c.table = np.tile(c.table, (1, 20))
    few = _rand((3, 4, 64), 5, DTYPES[dtype], 1.5)
    lists = torch.tensor(np.random.default_rng(3).integers(-1, c.table.shape[1], (3, 2, 300)), dtype=torch.int32).cuda()
    out = []
    for m in (300, 40, 3):
        i = torch.arange(m, device="cuda") % 3
        out.append(bl.attention_selected(few[i].contiguous(), c.cache, _i32(c.table).expand(m, -1).contiguous(), _i32([64 * 300] * m),
                                         lists[i].contiguous()))
    for many in out[:2]:
        for i in range(3):
            assert (many[i::3] == many[i]).all()
        off = (many[:3].float() - out[2].float()).abs().max() / out[2].float().abs().max()
        assert off < (2.0**-7 if dtype == "bf16" else 2e-5)


def test_selected_rows_that_are_not_finite(bl):  # noqa: F811
    c = _Paged(bl, [300], [3], 2, 64, 4)
    sel = np.tile(np.array([0, 2, 4]), (3, 2, 1))
    q, clean = _check_selected(bl, c, [300], [3], 8, sel, "f32")
    q[1, 2, 5], q[2, 7, 63] = float("nan"), float("inf")
    out = bl.attention_selected(q, c.cache, _i32(c.table), _i32([300]), _i32(sel), _starts([3])).view(3, 8, 64)
    bad = torch.zeros(3, 8, dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[2, 7] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean.view(3, 8, 64)[~bad])


def test_offsets_past_32_bits(bl):  # noqa: F811
    """Pages whose codes begin past 2^31 bytes: the prefix's, the bounds' and the chosen ones."""
    hkv, d = 8, 128
    pages = 2**31 // (hkv * 64 * d) + 40
    cache = bl.cache_alloc(pages, hkv, d)
    c = _Paged(bl, [300], [1], hkv, d, 6)
    far = pages - 1 - np.arange(c.pages)
    idx = torch.tensor(far, device="cuda")
    for big, small in zip(cache, c.cache):
        big[idx] = small
    table = _i32(far[c.table])
    q = _rand((1, 16, d), 1, torch.float32)
    near, lens = _i32(c.table), _i32([300])
    sel = _i32(np.tile(np.array([0, 3, 4]), (1, hkv, 1)))
    assert torch.equal(bl.attention_selected(q, cache, table, lens, sel), bl.attention_selected(q, c.cache, near, lens, sel))
    short = _i32([300 - 128])
    assert torch.equal(bl.attention_shared(q, cache, table[0, :2].contiguous(), _i32([128]), table[:, 2:].contiguous(), short),
                       bl.attention_shared(q, c.cache, near[0, :2].contiguous(), _i32([128]), near[:, 2:].contiguous(), short))
    bounds, small = bl.bounds_alloc(cache), bl.bounds_alloc(c.cache)
    bl.cache_bounds(cache, bounds, table, _i32([0]), _starts([300]), 300)
    bl.cache_bounds(c.cache, small, near, _i32([0]), _starts([300]), 300)
    assert torch.equal(bounds[idx], small)


# ---------------------------------------------------------------- the calls themselves

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_outside_the_sequences(bl, dtype):  # noqa: F811
    """Rows before the first and behind the last sequence, NaN among them: not written, and nothing of them enters."""
    c, prefix = _behind(bl)
    q = _rand((11, 8, 64), 3, DTYPES[dtype])
    inner = q[2:7].contiguous()
    q[:2], q[7:] = float("nan"), float("inf")
    table, lens, cu, inside = _i32(c.table), _i32([70, 3]), _i32([2, 4, 7]), _starts([2, 3])
    sel = _i32(np.random.default_rng(1).integers(-1, c.wide, (11, 2, 3)))
    bounds = bl.bounds_alloc(c.cache)
    bl.cache_bounds(c.cache, bounds, table, _i32([0, 0]), _starts([72, 6]), 78)
    for call, shape, fill in (
        (lambda x, s, o, off: bl.attention_shared(x, c.cache, _i32(prefix), _i32([150]), table, lens, off, out=o), (512,), 7.0),
        (lambda x, s, o, off: bl.attention_selected(x, c.cache, table, lens, s, off, out=o), (512,), 7.0),
        (lambda x, s, o, off: bl.block_select(x, bounds, c.cache.k_scale, table, lens, 1, off, out=o), (2, 1), 7),
    ):
        type_ = torch.int32 if isinstance(fill, int) else DTYPES[dtype]
        out = call(q, sel, torch.full((11, *shape), fill, dtype=type_, device="cuda"), cu)
        alone = call(inner, sel[2:7].contiguous(), torch.full((5, *shape), fill, dtype=type_, device="cuda"), inside)
        assert torch.equal(out[2:7], alone) and (out[:2] == fill).all() and (out[7:] == fill).all()


def test_binding_refusals(bl):  # noqa: F811
    """What the tensors themselves get wrong, before anything is enqueued."""
    q, k = _rand((6, 4, 64), 1, torch.bfloat16), _rand((6, 2, 64), 2, torch.bfloat16)
    cu, cache = _starts([6]), bl.cache_alloc(4, 2, 64)
    table, lens, f = _i32([[0, 1]]), _i32([3]), bl.rotary_frequencies(64)
    bounds, sel = bl.bounds_alloc(cache), _i32(np.zeros((6, 2, 3)))
    gain = torch.ones(64, device="cuda")
    for call in (
        lambda: bl.rotate(q.half(), k.half(), f, lens, cu), lambda: bl.rotate(q, k.float(), f, lens, cu), lambda: bl.rotate(q, k[:5], f, lens, cu),
        lambda: bl.rotate(q, k, f.double(), lens, cu), lambda: bl.rotate(q, k, f[:7].contiguous(), lens, cu), lambda: bl.rotate(q, k, f[:0], lens, cu),
        lambda: bl.rotate(q, k, f.view(2, 16), lens, cu), lambda: bl.rotate(q, k, f, lens), lambda: bl.rotate(q, k, f, lens.long(), cu),
        lambda: bl.rotate(q, k, f, lens, cu, q_gain=gain[:32].contiguous()), lambda: bl.rotate(q, k, f, lens, cu, k_gain=gain.bfloat16()),
        lambda: bl.rotate(q, k, f, lens, cu, eps=-1.0), lambda: bl.rotate(q, k, f, lens, cu, magnitude=float("nan")),
        lambda: bl.rotate(q, k, f, lens, cu, out=(q, q)), lambda: bl.rotate(q, k, f, lens, cu, out=q), lambda: bl.rotate(q, k, f, lens, cu, out=(q.float(), k)),
        lambda: bl.rotate(q, k, bl.rotary_frequencies(128), lens, cu), lambda: bl.rotate(q, k, f.cpu(), lens, cu),
        lambda: bl.attention_shared(q, cache, table, lens, table, lens, cu), lambda: bl.attention_shared(q, cache, table[0], _i32([1, 2]), table, lens, cu),
        lambda: bl.attention_shared(q, cache, table[0].long(), lens, table, lens, cu), lambda: bl.attention_shared(q, cache, table[0, :0], lens, table, lens, cu),
        lambda: bl.attention_shared(q, cache, table[0], lens, table, lens), lambda: bl.attention_shared(q, cache, table[0], lens, table, lens, cu, scale=float("inf")),
        lambda: bl.attention_shared(q, cache, table[0], lens, table, lens, cu, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
        lambda: bl.cache_bounds(cache, bounds[:3], table, lens, cu, 6), lambda: bl.cache_bounds(cache, bounds.float(), table, lens, cu, 6),
        lambda: bl.cache_bounds(cache, bounds, table, lens, None, 6), lambda: bl.cache_bounds(cache, bounds, table, lens, cu, 0),
        lambda: bl.block_select(q, bounds, cache.k_scale, table, lens, 0, cu), lambda: bl.block_select(q, bounds, cache.k_scale, table, lens, 2, cu, first=2),
        lambda: bl.block_select(q, bounds, cache.k_scale[:3], table, lens, 2, cu), lambda: bl.block_select(q, bounds[..., :32].contiguous(), cache.k_scale, table, lens, 2, cu),
        lambda: bl.block_select(_rand((6, 3, 64), 1, torch.bfloat16), bounds, cache.k_scale, table, lens, 2, cu),
        lambda: bl.block_select(q, bounds, cache.k_scale, table, lens, 2, cu, out=sel), lambda: bl.block_select(q, bounds, cache.k_scale, table, lens, 1 << 62, cu),
        lambda: bl.attention_selected(q, cache, table, lens, sel[:5], cu), lambda: bl.attention_selected(q, cache, table, lens, sel[:, :1], cu),
        lambda: bl.attention_selected(q, cache, table, lens, sel[..., :0], cu), lambda: bl.attention_selected(q, cache, table, lens, sel.long(), cu),
        lambda: bl.attention_selected(q, cache, table, lens, sel),
    ):
        with pytest.raises(bl.BitLinearError):
            call()
    with pytest.raises(TypeError):
        bl.rotate(q, k, f, lens, cu, eps="little")


def test_callers_workspaces(bl):  # noqa: F811
    c, prefix = _behind(bl, length=900)
    q = _rand((5, 8, 64), 1, torch.float32)
    args = (q, c.cache, _i32(prefix), _i32([900]), _i32(c.table), _i32([70, 3]), _starts([2, 3]))
    need = bl.attention_shared_workspace_size(5, 8, 2, 64, 2, c.wide, len(prefix))
    want = bl.attention_shared(*args)
    for n in (need, 2 * need):
        assert torch.equal(bl.attention_shared(*args, workspace=torch.full((n,), 255, dtype=torch.uint8, device="cuda")), want)
    c = _Paged(bl, [9000], [1], 2, 64, 8)
    sel = _i32(np.random.default_rng(1).integers(0, c.wide, (1, 2, 130)))
    need = bl.attention_selected_workspace_size(1, 8, 2, 64, 130)
    assert need > 0
    args = (q[:1], c.cache, _i32(c.table), _i32([9000]), sel)
    assert torch.equal(bl.attention_selected(*args, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda")), bl.attention_selected(*args))


class _Layer:
    """What a decode step of one layer does around its cache, the chosen and the whole attention over it."""

    def __init__(self, bl, dtype):  # noqa: F811
        self.bl, self.hq, self.hkv, self.d = bl, 8, 2, 64
        self.qkv = torch.zeros((3, (self.hq + 2 * self.hkv) * self.d), dtype=DTYPES[dtype], device="cuda")
        self.freq, self.gain = bl.rotary_frequencies(64, 10000.0), 1 + 0.1 * _rand((64,), 3, torch.float32)
        self.table = _i32(np.random.default_rng(2).permutation(60).reshape(3, 20))
        self.lens, self.begin, self.prefix_len = _i32([700, 20, 130]), _i32([900, 220, 330]), _i32([200])
        self.prefix = _i32([61, 60, 63, 62])

    def fresh(self):
        c = _Paged(self.bl, [64 * 64], [0], self.hkv, self.d, 9)
        return c.cache, self.bl.bounds_alloc(c.cache)

    def step(self, cache, bounds):
        q, k, v = (x.unflatten(1, (-1, self.d)) for x in self.qkv.split([self.hq * self.d, self.hkv * self.d, self.hkv * self.d], 1))
        q, k = self.bl.rotate(q, k, self.freq, self.begin, q_gain=self.gain, k_gain=self.gain)
        self.bl.cache_append(cache, k, v, self.table, self.lens)
        self.bl.cache_bounds(cache, bounds, self.table, self.lens, None, 3)
        sel = self.bl.block_select(q, bounds, cache.k_scale, self.table, self.lens, 5, first=1, recent=2)
        return (q, k, sel, self.bl.attention_selected(q, cache, self.table, self.lens, sel),
                self.bl.attention_shared(q, cache, self.prefix, self.prefix_len, self.table, self.lens))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_layers_step(bl, dtype):  # noqa: F811
    """Rotation, append, bounds, choice and attention one after the other, every one against its definition on what the
    one before gave."""
    layer = _Layer(bl, dtype)
    cache, bounds = layer.fresh()
    host = lambda: (cached_ref.natural(cache.k.cpu().numpy(), place[0]), cache.k_scale.cpu().numpy(),  # noqa: E731
                    cached_ref.natural(cache.v.cpu().numpy(), place[1]), cache.v_scale.cpu().numpy())
    place = cached_ref.code_places(layer.d)
    table, lens = layer.table.cpu().numpy(), layer.lens.tolist()
    bl.cache_bounds(cache, bounds, layer.table, _i32([0, 0, 0]), _starts(lens), sum(lens))  # of the tokens before
    mine = np.zeros(bounds.shape, np.int8)
    ref.cache_bounds(host()[0], mine, table, [0, 0, 0], np.cumsum([0] + lens), sum(lens))
    layer.qkv.copy_(_rand(layer.qkv.shape, 40, DTYPES[dtype]))
    q, k, sel, out, behind = layer.step(cache, bounds)
    ref.cache_bounds(host()[0], mine, table, lens, None, 3)
    np.testing.assert_array_equal(bounds.cpu().numpy(), mine)
    np.testing.assert_array_equal(sel.cpu().numpy(), ref.block_select(_np(q), mine, host()[1], table, lens, 5, None, 1, 2, 0))
    scale = layer.d ** -0.5
    want, spread, reach, grain = ref.attention_selected(_np(q), *host(), table, lens, sel.cpu().numpy(), None, scale)
    _assert_within(_np(out).reshape(want.shape), want, _tolerance(want, spread, reach, grain, 5, layer.d, dtype, False))
    want, spread, reach, grain = ref.attention_shared(_np(q), *host(), layer.prefix.cpu().numpy(), 200, table, lens, None, scale)
    _assert_within(_np(behind).reshape(want.shape), want, _tolerance(want, spread, reach, grain, 24, layer.d, dtype, True))


def test_captured_steps_follow_their_inputs(bl):  # noqa: F811
    """The step in one graph; each replay, on new inputs and lengths and with eager calls between, gives what eager calls give."""
    layer = _Layer(bl, "bf16")
    cache, bounds = layer.fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(cache, bounds)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = layer.step(cache, bounds)
    start = layer.fresh()
    for t, s in zip((*cache, bounds), (*start[0], start[1])):
        t.copy_(s)
    mirror = layer.fresh()
    for i in range(5):
        layer.qkv.copy_(_rand(layer.qkv.shape, 100 + i, torch.bfloat16))
        layer.lens.copy_(_i32([700 + i, 20 + 70 * i, 130 - 40 * i]))
        layer.begin.copy_(_i32([900 + i, 220, -1 if i == 2 else 7]))
        layer.prefix_len.copy_(_i32([(200, 0, 256, 63, 1)[i]]))
        if i == 2:
            layer.lens[2] = -1
        unused = layer.lens[2].item() < 0  # its row is as it was in each: compare the others
        g.replay()
        torch.cuda.synchronize()
        want = layer.step(*mirror)
        rows = 2 if unused else 3
        for n, (x, y) in enumerate(zip(captured, want)):
            assert torch.equal(x[:rows], y[:rows]), (i, n)
        if not unused:
            assert all(torch.equal(x, y) for x, y in zip((*cache, bounds), (*mirror[0], mirror[1])))
        else:
            for t, s in zip((*cache, bounds), (*mirror[0], mirror[1])):
                t.copy_(s)


def test_another_stream(bl):  # noqa: F811
    """Calls on streams of their own, twice at once, give what they give alone."""
    c, prefix = _behind(bl, length=900, lens=(300, 40), new=(1, 1))
    table, lens, pre, plen = _i32(c.table), _i32([300, 40]), _i32(prefix), _i32([900])
    f, sel = bl.rotary_frequencies(64), _i32(np.random.default_rng(1).integers(0, 5, (2, 2, 4)))
    bounds = _rand((c.pages, 2, 2, 64), 3, torch.float32, 40).to(torch.int8)
    q = [_rand((2, 8, 64), i, torch.bfloat16) for i in range(2)]
    k = _rand((2, 2, 64), 9, torch.bfloat16)

    def step(x):
        return (*bl.rotate(x, k, f, lens), bl.attention_shared(x, c.cache, pre, plen, table, lens), bl.block_select(x, bounds, c.cache.k_scale, table, lens, 2),
                bl.attention_selected(x, c.cache, table, lens, sel))
    alone = [step(x) for x in q]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(5):
        for s, x in zip(streams, q):
            with torch.cuda.stream(s):
                outs.append(step(x))
    torch.cuda.synchronize()
    for i, got in enumerate(outs):
        assert all(torch.equal(a, b) for a, b in zip(got, alone[i % 2]))


# ---------------------------------------------------------------- the launch rules' other sides

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_selected_long_lists_of_one_sequences_rows(bl, dtype):  # noqa: F811
    """Rows of one sequence whose lists are long together and share blocks: every row as in a batch of a few, and those
    as the definition has them."""
    c = _Paged(bl, [4096], [303], 2, 64, 8)
    rng = np.random.default_rng(3)
    sel = np.sort(rng.integers(0, 64, (3, 2, 64)), -1)
    _, _ = _check_selected(bl, c, [4096], [3], 4, sel, dtype)
    q = _rand((3, 4, 64), 5, DTYPES[dtype], 1.5)
    lists, table, lens = _i32(sel), _i32(c.table), _i32([4096])
    few = bl.attention_selected(q, c.cache, table, lens, lists, _starts([3]))
    for m in (303, 60):
        i = torch.arange(m, device="cuda") % 3
        many = bl.attention_selected(q[i].contiguous(), c.cache, table, lens, lists[i].contiguous(), _starts([m]))
        for r in range(3):
            assert (many[r::3] == many[r]).all()
        off = (many[:3].float() - few.float()).abs().max() / few.float().abs().max()
        assert off < (2.0**-7 if dtype == "bf16" else 2e-5)


@pytest.mark.parametrize("m,wide", [(130, 700), (40, 1400), (48, 1500), (97, 1500), (64, 2100), (97, 2100), (98, 2049), (97, 8192)])
def test_select_many_rows_of_wide_tables(bl, m, wide):  # noqa: F811
    """Two heads of so many rows and blocks that the scores are a launch of their own, and that they are not, with the keys
    of either size of workgroup: three rows against the definition, the others as these."""
    ends = [64 * wide - 1, 64 * (wide - 37) + 5, 64 * 520]
    c = _Bounds(bl, ends, [1] * 3, 2, 64, 3, wide=wide, pages=400)
    c.ks = (0.5 + 2 * np.random.default_rng(4).random(c.ks.shape)).astype(np.float32)
    q = _rand((3, 4, 64), 8, torch.bfloat16, 1.5)
    few = c.check(bl, q, ends, 40, None, 1, 2)
    i = torch.arange(m, device="cuda") % 3
    many = bl.block_select(q[i].contiguous(), torch.tensor(c.bounds).cuda(), torch.tensor(c.ks).cuda(), _i32(c.table)[i].contiguous(),
                           _i32(ends)[i].contiguous(), 40, first=1, recent=2)
    assert torch.equal(many, few[i])


def test_select_beside_rows_outside_the_sequences(bl):  # noqa: F811
    """Rows of NaN and infinities before and behind the sequences, where scores decide: not written, nothing of them enters."""
    lens, new, cu = [64 * 40 + 3, 64 * 25], [2, 3], _i32([2, 4, 7])
    c = _Bounds(bl, lens, new, 2, 64, 3)
    q = _rand((11, 8, 64), 3, torch.float32)
    inner = q[2:7].contiguous()
    q[:2], q[7:] = float("nan"), float("inf")
    want = c.check(bl, inner, lens, 9, _starts(new), 1, 2)
    got = c.check(bl, q, lens, 9, cu, 1, 2)
    assert torch.equal(got[2:7], want) and (got[:2] == 77).all() and (got[7:] == 77).all()
    assert (want[:, :, 1:] > 0).all() and not torch.equal(want[0, 0], want[0, 1])  # by scores, which differ


@pytest.mark.parametrize("m", [1714, 1715])
def test_rotate_waves_of_a_token(bl, m):  # noqa: F811
    """Seven rounds of heads by a wave each, and by one wave."""
    _check_rotate(bl, [m - 5, 0, 5], [3, 0, 900], 20, 5, 128, 64, "f32")
