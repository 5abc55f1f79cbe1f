"""Host side of the attention calls (no GPU needed): the status codes of invalid
arguments and the binding's own checks, before anything is enqueued; and the
oracle's pins."""
import ctypes
import os

import numpy as np
import pytest

from oracle import attention as ref

BL_OK, BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_DTYPE, BL_ERR_WORKSPACE, BL_ERR_HIP, BL_ERR_VALUE = range(8)
A, MIS, ODD = 0x10000, 0x10004, 0x10002  # fake device addresses, never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def bl():
    import bit_ternary_weight_bitlinear_amd as m
    from bit_ternary_weight_bitlinear_amd import build
    if not os.path.exists(m.library_path()):
        build.build()
    elif not os.path.exists(build.BINDING):
        build.build_binding()
    m.load_library()
    return m


def _call(fn, names, base, **change):
    args = dict(base, **change)
    return fn(*[args[n] for n in names.split()])


ATTENTION = "q qs k ks v vs dtype m hq hkv d cu seqs scale out ws wn st"
ATTENTION_OK = dict(q=A, qs=1024, k=A, ks=256, v=A, vs=256, dtype=1, m=10, hq=8, hkv=2, d=128, cu=A, seqs=2, scale=0.1, out=A, ws=None,
                    wn=0, st=None)


@pytest.mark.parametrize("change,status", [
    ({"q": None}, BL_ERR_NULL), ({"cu": None}, BL_ERR_NULL), ({"out": None}, BL_ERR_NULL), ({"dtype": 2}, BL_ERR_DTYPE),
    ({"m": 0}, BL_ERR_SHAPE), ({"m": (1 << 22) + 1}, BL_ERR_SHAPE), ({"hkv": 3}, BL_ERR_SHAPE), ({"hkv": 0}, BL_ERR_SHAPE),
    ({"hq": 0}, BL_ERR_SHAPE), ({"hq": 8192, "qs": 1 << 20}, BL_ERR_SHAPE), ({"d": 96}, BL_ERR_SHAPE), ({"d": 0}, BL_ERR_SHAPE),
    ({"seqs": 0}, BL_ERR_SHAPE), ({"seqs": -1}, BL_ERR_SHAPE), ({"qs": 1016}, BL_ERR_SHAPE), ({"ks": 1 << 31}, BL_ERR_SHAPE),
    ({"vs": 260}, BL_ERR_ALIGN), ({"q": MIS}, BL_ERR_ALIGN), ({"v": MIS}, BL_ERR_ALIGN), ({"out": MIS}, BL_ERR_ALIGN),
    ({"cu": ODD}, BL_ERR_ALIGN), ({"scale": NAN}, BL_ERR_VALUE), ({"scale": INF}, BL_ERR_VALUE), ({"scale": -INF}, BL_ERR_VALUE),
])
def test_attention_refusals(bl, change, status):
    assert _call(bl.load_library().bitlinear_attention, ATTENTION, ATTENTION_OK, **change) == status


APPEND = "k ks v vs dtype m hkv d cu lens seqs table wide kc vc kscale vscale pages st"
APPEND_OK = dict(k=A, ks=256, v=A, vs=256, dtype=1, m=4, hkv=2, d=128, cu=A, lens=A, seqs=2, table=A, wide=4, kc=A, vc=A, kscale=A,
                 vscale=A, pages=9, st=None)


@pytest.mark.parametrize("change,status", [
    ({n: None}, BL_ERR_NULL) for n in "k v lens table kc vc kscale vscale".split()] + [
    ({"dtype": -1}, BL_ERR_DTYPE), ({"cu": None}, BL_ERR_SHAPE), ({"wide": 0}, BL_ERR_SHAPE), ({"wide": (1 << 20) + 1}, BL_ERR_SHAPE),
    ({"pages": 0}, BL_ERR_SHAPE), ({"pages": 1 << 31}, BL_ERR_SHAPE), ({"d": 80}, BL_ERR_SHAPE), ({"ks": 255}, BL_ERR_SHAPE),
    ({"ks": 257}, BL_ERR_ALIGN), ({"dtype": 0, "ks": 258}, BL_ERR_ALIGN), ({"kc": MIS}, BL_ERR_ALIGN), ({"vscale": ODD}, BL_ERR_ALIGN),
    ({"lens": ODD}, BL_ERR_ALIGN), ({"table": ODD}, BL_ERR_ALIGN)])
def test_append_refusals(bl, change, status):
    assert _call(bl.load_library().bitlinear_cache_append, APPEND, APPEND_OK, **change) == status


READ = "kc vc kscale vscale pages table wide cu begin seqs dtype m hkv d ko vo st"
READ_OK = dict(kc=A, vc=A, kscale=A, vscale=A, pages=9, table=A, wide=4, cu=A, begin=A, seqs=2, dtype=0, m=4, hkv=2, d=64, ko=A, vo=A, st=None)


@pytest.mark.parametrize("change,status", [
    ({n: None}, BL_ERR_NULL) for n in "kc vc kscale vscale table begin ko vo".split()] + [
    ({"dtype": 3}, BL_ERR_DTYPE), ({"cu": None}, BL_ERR_SHAPE), ({"m": 0}, BL_ERR_SHAPE), ({"ko": MIS}, BL_ERR_ALIGN), ({"begin": ODD}, BL_ERR_ALIGN)])
def test_read_refusals(bl, change, status):
    assert _call(bl.load_library().bitlinear_cache_read, READ, READ_OK, **change) == status


CACHED = "q qs dtype m hq hkv d cu lens seqs table wide kc vc kscale vscale pages scale out w ws wn st"
CACHED_OK = dict(q=A, qs=1024, dtype=1, m=2, hq=8, hkv=2, d=128, cu=None, lens=A, seqs=2, table=A, wide=64, kc=A, vc=A, kscale=A, vscale=A,
                 pages=99, scale=0.1, out=A, w=None, ws=A, wn=1 << 30, st=None)


@pytest.mark.parametrize("change,status", [
    ({n: None}, BL_ERR_NULL) for n in "q lens table kc vc kscale vscale out ws".split()] + [
    ({"dtype": 9}, BL_ERR_DTYPE), ({"seqs": 3}, BL_ERR_SHAPE), ({"hkv": 5}, BL_ERR_SHAPE), ({"d": 256}, BL_ERR_SHAPE), ({"scale": NAN}, BL_ERR_VALUE),
    ({"q": MIS}, BL_ERR_ALIGN), ({"w": ODD}, BL_ERR_ALIGN), ({"ws": A + 16}, BL_ERR_ALIGN), ({"wn": 8}, BL_ERR_WORKSPACE)])
def test_cached_refusals(bl, change, status):
    assert _call(bl.load_library().bitlinear_attention_cached, CACHED, CACHED_OK, **change) == status


EVICT = "table lens w seqs wide keep first recent t2 l2 w2 gone count st"
EVICT_OK = dict(table=A, lens=A, w=A, seqs=2, wide=64, keep=8, first=1, recent=1, t2=A, l2=A, w2=A, gone=A, count=A, st=None)


@pytest.mark.parametrize("change,status", [
    ({n: None}, BL_ERR_NULL) for n in "table lens w t2 l2 w2 gone count".split()] + [
    ({"seqs": 0}, BL_ERR_SHAPE), ({"wide": 0}, BL_ERR_SHAPE), ({"first": -1}, BL_ERR_VALUE), ({"recent": 0}, BL_ERR_VALUE), ({"keep": 1}, BL_ERR_VALUE),
    ({"keep": 1 << 40, "recent": 1 << 62}, BL_ERR_VALUE), ({"w": ODD}, BL_ERR_ALIGN), ({"gone": ODD}, BL_ERR_ALIGN)])
def test_evict_refusals(bl, change, status):
    assert _call(bl.load_library().bitlinear_cache_evict, EVICT, EVICT_OK, **change) == status


def test_workspace_sizes(bl):
    import torch
    size = bl.attention_cached_workspace_size
    assert size(0, 8, 2, 128, 1, 64) == 0 and size(1, 8, 3, 128, 1, 64) == 0 and size(1, 8, 2, 100, 1, 64) == 0
    assert size(1, 32, 8, 128, 1, 2048) > 0                                    # one long sequence is split
    assert size(1024, 32, 8, 128, 1024, 2048) == 0                             # a large batch is not
    assert size(1024, 32, 8, 128, 1024, 2048, True) >= 1024 * 32 * 2048 * 8    # a value per row and block
    big = size(1 << 22, 4096, 1, 128, 1 << 22, 1 << 20, True)
    assert big > 1 << 57                                                       # the widest sizes do not wrap
    assert bl.attention_workspace_size(torch.int8, 8, 8, 2, 128, 1) == 0


def test_binding_refuses_host_tensors(bl):
    import torch
    x = torch.zeros((4, 2, 64))
    cu = torch.tensor([0, 4], dtype=torch.int32)
    cache = bl.cache_alloc(2, 2, 64, device="cpu")
    with pytest.raises(bl.BitLinearError):
        bl.attention(x, x, x, cu)
    with pytest.raises(bl.BitLinearError):
        bl.cache_append(cache, x, x, torch.zeros((1, 2), dtype=torch.int32), cu[:1], cu)
    with pytest.raises(bl.BitLinearError):
        bl.attention_cached(x, cache, torch.zeros((1, 2), dtype=torch.int32), cu[:1], cu)
    with pytest.raises(bl.BitLinearError):
        bl.cache_evict(torch.zeros((1, 2), dtype=torch.int32), cu[:1], torch.zeros((1, 2)), 1)
    with pytest.raises(bl.BitLinearError):
        bl.cache_alloc(2, 2, 96, device="cpu")


# ---------------------------------------------------------------- the oracle

def test_oracle_attention_by_hand():
    """Two keys of equal logits average; a third that is ln 2 higher takes half."""
    q = np.ones((3, 1, 1))
    k = np.array([0.0, 0.0, np.log(2)]).reshape(3, 1, 1)
    v = np.array([4.0, 8.0, 2.0]).reshape(3, 1, 1)
    out, spread, reach = ref.attention(q, k, v, [0, 3], 1.0)
    np.testing.assert_allclose(out.ravel(), [4, 6, 4], rtol=1e-15)
    out, *_ = ref.attention(q, k, v, [0, 1, 1, 3], 1.0)  # packed: the first row stands alone
    np.testing.assert_allclose(out.ravel(), [4, 8, 4], rtol=1e-15)


def test_oracle_append_by_hand():
    codes, scales = np.zeros((1, 1, 64, 4), np.int8), np.zeros((1, 1), np.float32)
    table = np.array([[0]])
    ref.cache_append(codes, scales, np.array([1.0, -2.0, 0.5, 0.0]).reshape(1, 1, 4), table, [0], None)
    assert scales[0, 0] == 2 and codes[0, 0, 0].tolist() == [64, -127, 32, 0]      # 63.5 to even, 31.75
    ref.cache_append(codes, scales, np.array([4.0, 1.0, 0.0, -4.0]).reshape(1, 1, 4), table, [1], None)
    assert scales[0, 0] == 4 and codes[0, 0, 1].tolist() == [127, 32, 0, -127]
    assert codes[0, 0, 0].tolist() == [32, -64, 16, 0]                             # halves; -63.5 to even
    values, there = ref.tokens(codes, scales, table[0], 0, 2)
    assert there.all() and values[1, 0, 0] == 4


def test_oracle_storage_rule_is_a_permutation():
    for d in (64, 128):
        for place in ref.code_places(d):
            assert sorted(place.ravel().tolist()) == list(range(64 * d))
    k, v = ref.code_places(128)
    assert (k[0, :16] == np.arange(16)).all() and (v[:16, 0] == np.arange(16)).all()   # 16 dims, 16 tokens adjacent
    assert k[4, 0] == 16 and k[1, 0] == 2048 and v[0, 1] == 16 and v[16, 0] == 256


def test_oracle_cached_agrees_with_the_prompt_form():
    rng = np.random.default_rng(1)
    n, hq, hkv, d = 70, 4, 2, 64
    kc, vc = (rng.integers(-127, 128, (2, hkv, 64, d)).astype(np.int8) for _ in range(2))
    ks, vs = (rng.random((2, hkv)).astype(np.float32) for _ in range(2))
    table = np.array([[1, 0]])
    k, v = (ref.tokens(c, s, table[0], 0, n)[0] for c, s in ((kc, ks), (vc, vs)))
    q = rng.standard_normal((n, hq, d))
    want, *_ = ref.attention(q, k, v, [0, n], 0.1)
    got, weights, *_ = ref.attention_cached(q, kc, ks, vc, vs, table, [0], [0, n], 0.1)
    np.testing.assert_allclose(got, want, rtol=1e-12)
    np.testing.assert_allclose(weights.sum(), n * hq, rtol=1e-12)


def test_oracle_evict_by_hand():
    table, lens = np.array([[10, 11, 12, 13, 14]], np.int32), np.array([290], np.int32)
    w = np.array([[1.0, 5.0, 2.0, 5.0, 0.0]], np.float32)
    t, n, kept, gone, count = ref.cache_evict(table, lens, w, 3, 1, 1)
    assert t.tolist() == [[10, 11, 14, -1, -1]] and n.tolist() == [290 - 128] and kept.tolist() == [[1, 5, 0, 0, 0]]
    assert gone.tolist() == [[12, 13, -1, -1, -1]] and count.tolist() == [2]
