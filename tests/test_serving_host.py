"""Host side of the position rotation, the shared prefix and the chosen blocks (no GPU needed): the status codes of
invalid arguments and the binding's own checks, before anything is enqueued; the frequencies; and the oracle's pins."""
import math

import numpy as np
import pytest

from oracle import attention as cached
from oracle import serving as ref
from tests.test_attention_host import (A, BL_ERR_ALIGN, BL_ERR_DTYPE, BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_VALUE, BL_ERR_WORKSPACE, INF, MIS, NAN,
                                       ODD, _call, bl)  # noqa: F401

ROTATE = "q qs k ks dtype m hq hkv d cu begin seqs freq rot inter mag qg kg eps qo qos ko kos st"
ROTATE_OK = dict(q=A, qs=1024, k=A, ks=256, dtype=1, m=10, hq=8, hkv=2, d=128, cu=A, begin=A, seqs=2, freq=A, rot=128, inter=0, mag=1.0, qg=None,
                 kg=None, eps=1e-5, qo=A, qos=1024, ko=A, kos=256, st=None)


@pytest.mark.parametrize("change,status", [
    ({n: None}, BL_ERR_NULL) for n in "q k begin freq qo ko".split()] + [
    ({"dtype": 2}, BL_ERR_DTYPE), ({"m": 0}, BL_ERR_SHAPE), ({"hkv": 3}, BL_ERR_SHAPE), ({"d": 96}, BL_ERR_SHAPE), ({"seqs": 0}, BL_ERR_SHAPE),
    ({"cu": None}, BL_ERR_SHAPE), ({"rot": 0}, BL_ERR_SHAPE), ({"rot": 8}, BL_ERR_SHAPE), ({"rot": 24}, BL_ERR_SHAPE), ({"rot": 144}, BL_ERR_SHAPE),
    ({"rot": -16}, BL_ERR_SHAPE), ({"d": 64, "rot": 128}, BL_ERR_SHAPE), ({"qs": 1016}, BL_ERR_SHAPE), ({"qos": 1016}, BL_ERR_SHAPE),
    ({"inter": 2}, BL_ERR_VALUE), ({"inter": -1}, BL_ERR_VALUE), ({"mag": NAN}, BL_ERR_VALUE), ({"mag": INF}, BL_ERR_VALUE),
    ({"eps": -1e-9}, BL_ERR_VALUE), ({"eps": NAN}, BL_ERR_VALUE), ({"ks": 260}, BL_ERR_ALIGN), ({"kos": 260}, BL_ERR_ALIGN), ({"q": MIS}, BL_ERR_ALIGN),
    ({"ko": MIS}, BL_ERR_ALIGN), ({"qg": MIS}, BL_ERR_ALIGN), ({"kg": MIS}, BL_ERR_ALIGN), ({"freq": ODD}, BL_ERR_ALIGN), ({"begin": ODD}, BL_ERR_ALIGN),
    ({"cu": ODD}, BL_ERR_ALIGN)])
def test_rotate_refusals(bl, change, status):  # noqa: F811
    assert _call(bl.load_library().bitlinear_rotate, ROTATE, ROTATE_OK, **change) == status


SHARED = "q qs dtype m hq hkv d pt pb pl cu lens seqs table wide kc vc kscale vscale pages scale out ws wn st"
SHARED_OK = dict(q=A, qs=1024, dtype=1, m=2, hq=8, hkv=2, d=128, pt=A, pb=32, pl=A, cu=None, lens=A, seqs=2, table=A, wide=64, kc=A, vc=A,
                 kscale=A, vscale=A, pages=99, scale=0.1, out=A, ws=A, wn=1 << 30, st=None)


@pytest.mark.parametrize("change,status", [
    ({n: None}, BL_ERR_NULL) for n in "q pt pl lens table kc vc kscale vscale out ws".split()] + [
    ({"dtype": 9}, BL_ERR_DTYPE), ({"seqs": 3}, BL_ERR_SHAPE), ({"hkv": 5}, BL_ERR_SHAPE), ({"d": 256}, BL_ERR_SHAPE), ({"pb": 0}, BL_ERR_SHAPE),
    ({"pb": (1 << 20) + 1}, BL_ERR_SHAPE), ({"m": 1 << 22, "seqs": 1 << 22, "hq": 4096, "hkv": 1, "d": 64, "qs": 1 << 18}, BL_ERR_SHAPE),
    ({"scale": NAN}, BL_ERR_VALUE), ({"q": MIS}, BL_ERR_ALIGN), ({"pt": ODD}, BL_ERR_ALIGN), ({"pl": ODD}, BL_ERR_ALIGN), ({"ws": A + 16}, BL_ERR_ALIGN),
    ({"wn": 8}, BL_ERR_WORKSPACE)])
def test_shared_refusals(bl, change, status):  # noqa: F811
    assert _call(bl.load_library().bitlinear_attention_shared, SHARED, SHARED_OK, **change) == status


BOUNDS = "kc pages hkv d m cu lens seqs table wide bounds st"
BOUNDS_OK = dict(kc=A, pages=9, hkv=2, d=128, m=4, cu=A, lens=A, seqs=2, table=A, wide=4, bounds=A, st=None)


@pytest.mark.parametrize("change,status", [
    ({n: None}, BL_ERR_NULL) for n in "kc lens table bounds".split()] + [
    ({"m": 0}, BL_ERR_SHAPE), ({"cu": None}, BL_ERR_SHAPE), ({"pages": 1 << 31}, BL_ERR_SHAPE), ({"d": 80}, BL_ERR_SHAPE), ({"wide": 0}, BL_ERR_SHAPE),
    ({"kc": MIS}, BL_ERR_ALIGN), ({"bounds": MIS}, BL_ERR_ALIGN), ({"lens": ODD}, BL_ERR_ALIGN)])
def test_bounds_refusals(bl, change, status):  # noqa: F811
    assert _call(bl.load_library().bitlinear_cache_bounds, BOUNDS, BOUNDS_OK, **change) == status


SELECT = "q qs dtype m hq hkv d cu lens seqs table wide bounds kscale pages keep first recent out ws wn st"
SELECT_OK = dict(q=A, qs=1024, dtype=0, m=2, hq=8, hkv=2, d=128, cu=None, lens=A, seqs=2, table=A, wide=20000, bounds=A, kscale=A, pages=99, keep=8,
                 first=1, recent=2, out=A, ws=A, wn=1 << 30, st=None)


@pytest.mark.parametrize("change,status", [
    ({n: None}, BL_ERR_NULL) for n in "q lens table bounds kscale out ws".split()] + [
    ({"dtype": 9}, BL_ERR_DTYPE), ({"seqs": 3}, BL_ERR_SHAPE), ({"hq": 129, "hkv": 1, "qs": 1 << 15}, BL_ERR_SHAPE), ({"wide": 0}, BL_ERR_SHAPE),
    ({"first": -1}, BL_ERR_VALUE), ({"recent": 0}, BL_ERR_VALUE), ({"keep": 2}, BL_ERR_VALUE), ({"keep": (1 << 20) + 1}, BL_ERR_VALUE),
    ({"keep": 1 << 40, "recent": 1 << 62}, BL_ERR_VALUE), ({"bounds": MIS}, BL_ERR_ALIGN), ({"out": ODD}, BL_ERR_ALIGN), ({"wn": 8}, BL_ERR_WORKSPACE)])
def test_select_refusals(bl, change, status):  # noqa: F811
    assert _call(bl.load_library().bitlinear_block_select, SELECT, SELECT_OK, **change) == status


SELECTED = "q qs dtype m hq hkv d cu lens seqs table wide sel keep kc vc kscale vscale pages scale out ws wn st"
SELECTED_OK = dict(q=A, qs=1024, dtype=1, m=2, hq=8, hkv=2, d=128, cu=None, lens=A, seqs=2, table=A, wide=64, sel=A, keep=300, kc=A, vc=A, kscale=A,
                   vscale=A, pages=99, scale=0.1, out=A, ws=A, wn=1 << 30, st=None)


@pytest.mark.parametrize("change,status", [
    ({n: None}, BL_ERR_NULL) for n in "q lens table sel kc vc kscale vscale out ws".split()] + [
    ({"dtype": 9}, BL_ERR_DTYPE), ({"seqs": 3}, BL_ERR_SHAPE), ({"keep": 0}, BL_ERR_SHAPE), ({"keep": (1 << 20) + 1}, BL_ERR_SHAPE),
    ({"m": 1 << 22, "seqs": 1 << 22, "hq": 4096, "hkv": 1, "d": 64, "qs": 1 << 18}, BL_ERR_SHAPE), ({"scale": INF}, BL_ERR_VALUE),
    ({"sel": ODD}, BL_ERR_ALIGN), ({"out": MIS}, BL_ERR_ALIGN), ({"wn": 8}, BL_ERR_WORKSPACE)])
def test_selected_refusals(bl, change, status):  # noqa: F811
    assert _call(bl.load_library().bitlinear_attention_selected, SELECTED, SELECTED_OK, **change) == status


def test_workspace_sizes(bl):  # noqa: F811
    assert bl.attention_shared_workspace_size(0, 8, 2, 128, 1, 4, 4) == 0 and bl.attention_shared_workspace_size(1, 8, 2, 128, 1, 4, 0) == 0
    assert bl.attention_shared_workspace_size(64, 32, 8, 128, 64, 32, 256) >= 64 * 32 * 130 * 4
    assert bl.attention_shared_workspace_size(1 << 18, 4096, 1, 128, 1 << 18, 1 << 20, 1 << 20) >= (1 << 30) * 130 * 4  # does not wrap
    assert bl.block_select_workspace_size(64, 8, 2048) == 0 and bl.block_select_workspace_size(1, 8, 2048) == 8 * 4 * 2048 and bl.block_select_workspace_size(7, 8, 1 << 20) == 7 * 8 * 4 << 20
    assert bl.block_select_workspace_size(1, 0, 1 << 20) == 0
    assert bl.attention_selected_workspace_size(1, 32, 8, 128, 64) > 0 and bl.attention_selected_workspace_size(1024, 32, 8, 128, 64) == 0
    assert bl.attention_selected_workspace_size(1, 32, 8, 96, 64) == 0


def test_binding_refuses_host_tensors(bl):  # noqa: F811
    import torch
    q, k = torch.zeros((4, 4, 64)), torch.zeros((4, 2, 64))
    cu, i32 = torch.tensor([0, 4], dtype=torch.int32), torch.zeros((1, 2), dtype=torch.int32)
    cache = bl.cache_alloc(2, 2, 64, device="cpu")
    bounds = bl.bounds_alloc(cache)
    assert bounds.shape == (2, 2, 2, 64) and bounds.dtype == torch.int8
    for call in (lambda: bl.rotate(q, k, bl.rotary_frequencies(64, device="cpu"), cu[:1], cu),
                 lambda: bl.attention_shared(q, cache, i32[0], cu[:1], i32, cu[:1], cu), lambda: bl.cache_bounds(cache, bounds, i32, cu[:1], cu, 4),
                 lambda: bl.block_select(q, bounds, cache.k_scale, i32, cu[:1], 1, cu),
                 lambda: bl.attention_selected(q, cache, i32, cu[:1], torch.zeros((4, 2, 1), dtype=torch.int32), cu)):
        with pytest.raises(bl.BitLinearError):
            call()


# ---------------------------------------------------------------- frequencies

def test_frequencies(bl):  # noqa: F811
    f = bl.rotary_frequencies(64, 10000.0, device="cpu").double()
    assert f.dtype != f.float().dtype and f.shape == (32,) and f[0] == 1
    np.testing.assert_allclose(f[16].item(), 0.01, rtol=2**-24)             # half way down from 1 to 1 / base
    np.testing.assert_allclose(bl.rotary_frequencies(64, 10000.0, scaling="positions", factor=4.0, device="cpu").double(), f / 4, rtol=2**-23)
    base = bl.rotary_frequencies(64, 10000.0, scaling="base", factor=4.0, device="cpu").double()
    assert base[0] == 1
    np.testing.assert_allclose(base[31].item(), f[31].item() / 4, rtol=2**-22)  # the slowest pair: divided by the factor
    assert (base[1:] < f[1:]).all() and (base > f / 4.0000001).all()
    part = bl.rotary_frequencies(64, 10000.0, scaling="parts", factor=8.0, length=4096, low=1, high=32, device="cpu").double()
    turns = 4096 * f / (2 * math.pi)
    assert (turns > 32).any() and (turns < 1).any()
    np.testing.assert_array_equal(part[turns > 32.01], f[turns > 32.01])
    np.testing.assert_allclose(part[turns < 0.99], f[turns < 0.99] / 8, rtol=2**-23)
    middle = (turns > 1.01) & (turns < 31.9)
    share = (turns[middle] - 1) / 31
    np.testing.assert_allclose(part[middle], f[middle] * (share + (1 - share) / 8), rtol=2**-21)


@pytest.mark.parametrize("args,kw", [((0,), {}), ((24,), {}), ((64, 0.0), {}), ((64, INF), {}), ((64,), {"scaling": "most"}), ((64,), {"scaling": "parts"}),
                                     ((64,), {"scaling": "parts", "length": 9, "low": 4.0, "high": 4.0}), ((64,), {"factor": 0.0}), ((64,), {"factor": NAN})])
def test_frequencies_refused(bl, args, kw):  # noqa: F811
    with pytest.raises(bl.BitLinearError):
        bl.rotary_frequencies(*args, device="cpu", **kw)


# ---------------------------------------------------------------- the oracle

def test_oracle_rotate_by_hand():
    """A quarter turn per position: (a, b) -> (-b, a) -> (-a, -b); the third element pair stays."""
    x = np.array([1.0, 2.0, 3.0, 4.0, 5.0, 6.0]).reshape(1, 1, 6).repeat(3, 0)
    half, _ = ref.rotate(x, [0, 1, 2], [np.pi / 2, 0.0], False, None, 0, 1.0)
    np.testing.assert_allclose(half[:, 0], [[1, 2, 3, 4, 5, 6], [-3, 2, 1, 4, 5, 6], [-1, 2, -3, 4, 5, 6]], atol=1e-14)
    turned, size = ref.rotate(x, [0, 1, 2], [np.pi / 2, 0.0], True, None, 0, 2.0)
    np.testing.assert_allclose(turned[:, 0], [[2, 4, 6, 8, 5, 6], [-4, 2, 6, 8, 5, 6], [-2, -4, 6, 8, 5, 6]], atol=1e-14)
    assert size[0, 0].tolist() == [3, 3, 7, 7, 5, 6]
    normed, _ = ref.rotate(np.array([3.0, 4.0]).reshape(1, 1, 2), [0], [1.0], True, [1.0, 0.5], 12.5, 1.0)  # mean square 12.5
    np.testing.assert_allclose(normed.ravel(), [0.6, 0.4])
    assert ref.positions([5, -1, 0], [1, 3, 4, 6], 8).tolist() == [-1, 5, 6, -1, 0, 1, -1, -1]


def test_oracle_rotation_keeps_products_of_equal_distances():
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((2, 1, 1, 64))
    f = 10000.0 ** (-np.arange(32) / 32)
    for inter in (False, True):
        dots = [float((ref.rotate(q, [n + 7], f, inter, None, 0, 1.0)[0] * ref.rotate(k, [n], f, inter, None, 0, 1.0)[0]).sum()) for n in (0, 1, 900)]
        np.testing.assert_allclose(dots, dots[0], rtol=1e-12)


def _cache(rng, pages, heads, d):
    codes = [rng.integers(-127, 128, (pages, heads, 64, d)).astype(np.int8) for _ in range(2)]
    scales = [rng.random((pages, heads)).astype(np.float32) + 0.5 for _ in range(2)]
    return codes[0], scales[0], codes[1], scales[1]


def test_oracle_shared_is_one_softmax():
    """A prefix of whole blocks and a sequence behind it: the same as one sequence that holds both."""
    rng = np.random.default_rng(5)
    c = _cache(rng, 6, 2, 64)
    q = rng.standard_normal((3, 4, 64))
    got, spread, reach, grain = ref.attention_shared(q, *c, [4, 1], 128, np.array([[0, 5]]), [70], [0, 3], 0.1)
    want, _, spread2, reach2, grain2 = cached.attention_cached(q, *c, np.array([[4, 1, 0, 5]]), [198], [0, 3], 0.1)
    for a, b in ((got, want), (spread, spread2), (reach, reach2), (grain, grain2)):
        np.testing.assert_allclose(a, b, rtol=1e-12)
    short, *_ = ref.attention_shared(q, *c, [4, 1], 0, np.array([[0, 5]]), [70], [0, 3], 0.1)  # no prefix
    np.testing.assert_allclose(short, cached.attention_cached(q, *c, np.array([[0, 5]]), [70], [0, 3], 0.1)[0], rtol=1e-12)


def test_oracle_selected_all_blocks_is_the_whole_cache():
    rng = np.random.default_rng(6)
    c = _cache(rng, 5, 2, 64)
    q, table = rng.standard_normal((2, 4, 64)), np.array([[3, 0, 4], [1, 2, -1]])
    sel = np.array([[[0, 1, 2]] * 2, [[1, -1, 0]] * 2])
    got = ref.attention_selected(q, *c, table, [150, 100], sel, None, 0.1)
    want = cached.attention_cached(q, *c, table, [150, 100], None, 0.1)
    np.testing.assert_allclose(got[0], want[0], rtol=1e-12)
    np.testing.assert_allclose(got[3], want[4], rtol=1e-12)
    twice = ref.attention_selected(q[:1], *c, table[:1], [150], np.array([[[0, 0]] * 2]), None, 0.1)
    once = ref.attention_selected(q[:1], *c, table[:1], [150], np.array([[[0]] * 2]), None, 0.1)
    np.testing.assert_allclose(twice[0], once[0], rtol=1e-12)  # every token twice: the same mean


def test_oracle_bounds_and_choice_by_hand():
    kc = np.zeros((3, 1, 64, 2), np.int8)
    kc[0, 0, :2] = [[3, -5], [-1, 7]]
    kc[0, 0, 2] = [100, 100]  # behind the last token
    bounds = np.full((3, 1, 2, 2), 9, np.int8)
    ref.cache_bounds(kc, bounds, np.array([[1, 0]]), [64], [0, 2], 2)
    assert bounds[0, 0].tolist() == [[3, 7], [-1, -5]] and (bounds[1:] == 9).all()
    # two heads (127, -127) and (0, 64): P = (127, 64), N = (0, -127)
    q = np.array([[[2.0, -2.0], [0.0, 1.0]]])  # 63.5 to even
    bounds = np.array([[[[3, 7], [-1, -5]]], [[[10, 0], [10, 0]]], [[[0, 0], [0, -20]]]], np.int8)
    # T = 127*3 + 64*7 + 127*5 = 1464; 1270; 127*20 = 2540
    ks = np.array([[1.0], [2.0], [0.5]], np.float32)  # scores 1464, 2540, 1270
    table = np.array([[0, 1, 2, 0, 1]])
    assert ref.block_select(q, bounds, ks, table, [319], 2, None, 0, 1, 7).tolist() == [[[1, 4]]]
    assert ref.block_select(q, bounds, ks, table, [319], 3, None, 0, 1, 7).tolist() == [[[0, 1, 4]]]     # of 0 and 3 the lower
    assert ref.block_select(q, bounds, ks, table, [319], 4, None, 1, 2, 7).tolist() == [[[0, 1, 3, 4]]]
    assert ref.block_select(q, bounds, ks, table, [70], 4, None, 0, 1, 7).tolist() == [[[0, 1, -1, -1]]]
    assert ref.block_select(q, bounds, ks, table, [-1], 1, None, 0, 1, 7).tolist() == [[[7]]]
