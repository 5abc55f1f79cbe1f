"""Attention behind a shared prefix at the ends of fp32's range: logits beyond fp32's integers, infinities that the cache
holds as the largest finite number. The inputs are such that the logits in powers of two are exact in fp32 (integers times
a power of two, scale * log2 e rounding to 1), so the weights are known: 2^(x - the largest x)."""
import math

import numpy as np
import pytest

from oracle import attention as cached_ref
from tests.test_attention import DTYPES, _assert_within, _i32, _np, _rand, _starts, bl, torch  # noqa: F401
from tests.test_serving import _behind

pytestmark = pytest.mark.gpu

LN2 = float(np.float32(0.6931472))  # times log2 e it rounds to 1
HALF = {"bf16": 2.0**-8, "f32": 2.0**-24}  # of a result's step
WEIGHT = {"bf16": 2.0**-11, "f32": 2.0**-22}  # of the weights over the prefix


def _set(codes, mine, place):
    codes.copy_(torch.tensor(cached_ref.stored(mine, place)))


def _scales(c, k):
    c.ks[:] = k
    c.cache.k_scale.copy_(torch.tensor(c.ks))


def _exact_logits(bl, sign, power, own_first, length=700, lens=(70, 3), new=(2, 3), d=64):  # noqa: F811
    """A cache whose keys meet a query of +-2^16 in dim 0 and 1 in dim 1 as +-127 * 2^16 + (a code of 0 to 3), times
    2^power; the own pages' first codes make them less than that by 2^16 times what own_first lacks of 127, or more."""
    c, prefix = _behind(bl, length=length, lens=lens, new=new, d=d)
    rng = np.random.default_rng(11)
    c.kc[:] = 0
    c.kc[..., 1] = rng.integers(0, 4, c.kc.shape[:3])
    first = np.full(c.pages, own_first)
    first[prefix] = 126
    c.kc[..., 0] = (sign * first)[:, None, None]
    _set(c.cache.k, c.kc, c.place[0])
    _scales(c, np.float32(127) * np.float32(2.0**power))  # a code stands for 2^power
    q = torch.zeros((sum(new), 8, d), device="cuda")
    q[:, :, 0], q[:, :, 1] = sign * 2.0**16, 1.0
    return c, prefix, q


def _call(bl, c, prefix, length, q, scale, lens=(70, 3), new=(2, 3)):  # noqa: F811
    return bl.attention_shared(q, c.cache, _i32(prefix), _i32([length]), _i32(c.table), _i32(lens), _starts(new), scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("negative", [False, True])
@pytest.mark.parametrize("power", [-10, -2, -1, 0, 1, 3, 4, 5, 8, 40, 90])
def test_shared_weights_beside_large_logits(bl, power, negative, d, dtype):  # noqa: F811
    """Logits near +-2^(23 + power), equal to some bits between tokens of many pages: their weights are as those of small
    logits. What the own pages hold has none. Per element: the weights' rounding of `spread`, the same again by their sum,
    700 additions and the joins of u = 2^-24 each, the result's own half step."""
    sign = -1 if negative else 1
    # the largest logits are the prefix's: own codes are below it, or the other way round where all are negative
    c, prefix, q = _exact_logits(bl, 1, power, 127 if negative else 100, d=d)
    q[:, :, 0] *= sign
    scale = LN2
    got = _np(_call(bl, c, prefix, 700, q.to(DTYPES[dtype]), scale)).reshape(5, 8, d)
    x = c.kc[prefix][..., 1].astype(np.float64)  # [blocks][heads][64]
    p = np.exp2((x - x.max()) * 2.0**power) if power < 10 else (x == x.max()).astype(np.float64)
    p = p.swapaxes(0, 1).reshape(2, -1)[:, :700]
    v = (c.vc[prefix].astype(np.float64) * (c.vs[prefix].astype(np.float64) / 127)[..., None, None]).swapaxes(0, 1).reshape(2, -1, d)[:, :700]
    want = np.einsum("hn,hnd->hd", p, v) / p.sum(1, keepdims=True)
    spread = np.einsum("hn,hnd->hd", p, np.abs(v)) / p.sum(1, keepdims=True)
    want, spread = (np.repeat(t, 4, 0)[None] for t in (want, spread))
    tol = 2 * (1.01 * WEIGHT[dtype] + 800 * 2.0**-24) * spread + HALF[dtype] * np.abs(want) + 1e-30
    _assert_within(got, np.broadcast_to(want, got.shape), np.broadcast_to(tol, got.shape), f"{power}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["prefix", "own"])
@pytest.mark.parametrize("negative", [False, True])
@pytest.mark.parametrize("power", [-8, -2, 3, 4, 7, 30, 77, 100])
def test_shared_one_key_takes_all(bl, power, negative, where, dtype):  # noqa: F811
    """Logits of up to 2^(23 + power) of either sign, K scales of 2^7 times 2^power: one token of the prefix, or the
    first own one, is above the rest by a hundredth of that, and the result is its V."""
    c, prefix = _behind(bl, length=640)
    rng = np.random.default_rng(12)
    c.kc[:] = 0
    c.kc[..., 0] = rng.integers(60, 101, c.kc.shape[:3])
    peak = 2 if negative else 127  # the row's largest logit, where q is negative the one nearest 0
    page = [int(prefix[7])] * 2 if where == "prefix" else [int(c.table[s, 0]) for s in (0, 1)]
    token = 33 if where == "prefix" else 0
    for i in page:
        c.kc[i, :, token, 0] = peak
    _set(c.cache.k, c.kc, c.place[0])
    _scales(c, np.float32(127) * np.float32(2.0**power))
    q = torch.zeros((5, 8, 64), device="cuda")
    q[:, :, 0] = (-1 if negative else 1) * 2.0**16
    for turn in (1, -1):  # scales of both signs
        got = _np(_call(bl, c, prefix, 640, (turn * q).to(DTYPES[dtype]), turn * LN2)).reshape(5, 8, 64)
        want = np.zeros((5, 8, 64))
        for r in range(5):
            i = page[0 if r < 2 else 1]
            v = c.vc[i, :, token].astype(np.float64) * (c.vs[i].astype(np.float64) / 127)[:, None]
            want[r] = np.repeat(v, 4, 0)
        # one weight, its digits or its rounding 2^-22 at most, a handful of roundings of u
        tol = (2.0**-20 + HALF[dtype]) * np.abs(want) + 1e-30
        _assert_within(got, want, tol, f"{power} {where} {turn}")


def _split(bl, k, v, table, pages, m, hkv, d):  # noqa: F811
    cache = bl.cache_alloc(pages, hkv, d)
    bl.cache_append(cache, k, v, table, _i32([0]), _starts([m]))
    return cache


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf])
def test_shared_infinite_keys(bl, bad, dtype):  # noqa: F811
    """An infinity of K, which the cache holds as the largest finite number: it takes the rows that have its sign there
    (their result is its V), the others give it nothing, as in attention over the whole cache."""
    hkv, d, n = 2, 64, 500
    k, v = (_rand((n, hkv, d), i, DTYPES[dtype]) for i in (1, 2))
    k[200, :, 5] = bad
    table = _i32(np.random.default_rng(1).permutation(8)[None])
    cache = _split(bl, k, v, table, 8, n, hkv, d)
    q = _rand((1, 8, d), 3, DTYPES[dtype])
    q[0, :, 5] = torch.tensor([1.0, -1.0] * 4)
    got = bl.attention_shared(q, cache, table[0, :6].contiguous(), _i32([384]), table[:, 6:].contiguous(), _i32([n - 1 - 384]))
    whole = bl.attention_cached(q, cache, table, _i32([n - 1]))
    np.testing.assert_allclose(_np(got), _np(whole), rtol=2**-7 if dtype == "bf16" else 2e-5, atol=(2**-8 if dtype == "bf16" else 2e-5) * float(whole.abs().max()))
    held = bl.cache_read(cache, table, _i32([200]), _starts([1]), 1, torch.float32)[1][0]
    takes = range(0, 8, 2) if bad > 0 else range(1, 8, 2)
    for h in takes:
        off = (got.view(8, d)[h].float() - held[h // 4]).abs()
        assert (off <= (2.0**-20 + HALF[dtype]) * held[h // 4].abs() + 1e-30).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, 1e37])
def test_shared_infinite_values(bl, bad, dtype):  # noqa: F811
    """An infinity of V, held as the largest finite number, and a large one: what the other dims hold is theirs still, as in
    attention over the whole cache."""
    hkv, d, n = 2, 64, 500
    k, v = (_rand((n, hkv, d), i, DTYPES[dtype]) for i in (1, 2))
    v[200, :, 5] = bad
    table = _i32(np.random.default_rng(1).permutation(8)[None])
    cache = _split(bl, k, v, table, 8, n, hkv, d)
    q = _rand((1, 8, d), 3, DTYPES[dtype])
    got = bl.attention_shared(q, cache, table[0, :6].contiguous(), _i32([384]), table[:, 6:].contiguous(), _i32([n - 1 - 384])).view(8, d)
    whole = bl.attention_cached(q, cache, table, _i32([n - 1])).view(8, d)
    rest = torch.arange(d, device="cuda") != 5
    assert torch.isfinite(whole[:, rest]).all()
    rel = 2**-7 if dtype == "bf16" else 2e-5
    np.testing.assert_allclose(_np(got)[:, rest.cpu().numpy()], _np(whole)[:, rest.cpu().numpy()], rtol=rel, atol=rel * float(whole[:, rest].abs().max()))
    np.testing.assert_allclose(_np(got)[:, 5], _np(whole)[:, 5], rtol=rel)


def test_shared_more_rows_than_one_launch_joins(bl):  # noqa: F811
    """2^25 query rows of 128, which are joined by a thread per element: every row as in a batch of four tokens."""
    m, hq, hkv, d = 2**19, 64, 8, 128
    if torch.cuda.get_device_properties(0).total_memory < 100e9:
        pytest.skip("needs 52 GB")
    c, prefix = _behind(bl, length=50, lens=(1000,), new=(4,), hkv=hkv, d=d)
    table = _i32(c.table[:, :1])  # the tokens past it do not exist: every row sees the same
    few = _rand((4, hq, d), 5, torch.bfloat16, 1.5)
    args = (c.cache, _i32(prefix[:1]), _i32([50]), table, _i32([1000]))
    want = bl.attention_shared(few, *args, _starts([4]))
    out = bl.attention_shared(few.repeat(m // 4, 1, 1), *args, _starts([m])).view(-1, 4, hq * d)
    for part in out.split(2**14):
        assert (part == out[0]).all()
    assert (out[0].float() - want.float()).abs().max() <= 2.0**-7 * want.float().abs().max()
    del out
    torch.cuda.empty_cache()
