"""Attention over the cache in every form of its kernel: 4, 8 and 16 query rows per workgroup, 4, 8 and 16 waves, one
workgroup per sequence and head or several joined by either joining kernel, and waves with more than 64 pages (a second
round of page ids and scales). The host's rule is mirrored here and each case says which form it is there for, so that a
changed rule fails test_forms instead of leaving one untested."""
import os

import numpy as np
import pytest

from oracle import attention as ref
from tests.test_attention import DTYPES, _assert_within, _i32, _np, _Paged, _rand, _starts, bl, torch  # noqa: F401

FEW = 16  # splits that a thread per dim joins by itself


def up(a, b):
    return -(-a // b)


def form(seqs, m, hq, hkv, d, wide):
    """(row tiles, waves, splits) that the host picks."""
    rows = up(m * (hq // hkv), seqs)
    units = lambda rt: seqs * up(rows, 4 * rt) * hkv  # noqa: E731
    pages = wide * d // 64
    if rows <= 4:
        rt = 1
    elif rows > 8 and units(4) * pages >= 20000:
        rt = 4
    else:
        rt = 1 if units(1) <= 256 and units(1) * pages <= 12000 else 2
    n = units(rt)
    lengthy = wide * d > 256 * 16 // rt
    waves = 16 // rt if n <= 256 or (lengthy and 2 * n >= 768 and n < 512) else 4
    if wide * d <= 256 * waves:
        return rt, waves, 1
    s = min((16 if rt == 1 else 8) * 256 // (waves * n), up(wide, waves))
    return rt, waves, 1 if n >= 512 or s < 1 else min(s, 256)


def parts(pages, splits, waves):
    """Workgroups that have pages of a sequence."""
    return up(pages, max(up(pages, splits), waves))


# lens, new, hq, hkv, d, blocks of the table, and (row tiles, waves, splits of more than one: joined by which kernel)
LONG = [([17 * 1024 + 300], [1]), ([20000, 70], [1, 1])]
CASES = [
    # 4 rows per workgroup
    ([1000, 5, 300], [1] * 3, 8, 2, 128, 16, (1, 16, "one")),
    ([5000, 64, 1], [1, 2, 1], 4, 2, 64, 90, (1, 16, "few")),
    (LONG[0][0], LONG[0][1], 4, 1, 128, 400, (1, 16, "many")),
    (LONG[1][0], LONG[1][1], 8, 2, 64, 400, (1, 16, "many")),
    ([30] * 129 + [20000], [1] * 130, 8, 2, 64, 320, (1, 4, "few")),
    ([40] * 255 + [17000, 33], [1] * 257, 4, 2, 64, 300, (1, 4, "one")),
    # 8 rows
    ([90, 4000, 7, 1300], [4] * 4, 20, 5, 128, 400, (2, 8, "few")),
    ([90, 4000, 7, 130] * 3, [4] * 12, 20, 5, 128, 63, (2, 8, "few")),
    ([150, 63, 0, 64, 200] * 40, [1] * 200, 8, 1, 64, 8, (2, 8, "one")),
    ([18000, 100], [1, 1], 8, 1, 128, 3100, (2, 8, "many")),
    ([18000, 100], [2, 3], 6, 2, 64, 3100, (2, 8, "many")),
    ([50] * 150 + [34000], [1] * 151, 8, 1, 64, 540, (2, 8, "one")),
    ([20, 300, 64] * 100, [2] * 300, 8, 2, 64, 6, (2, 4, "one")),
    ([50] * 270 + [17000], [1] * 271, 8, 1, 128, 270, (2, 4, "one")),
    # 16 rows
    ([100, 1500, 0], [8, 3, 12], 32, 8, 128, 256, (4, 4, "few")),
    ([3000, 100], [6, 10], 32, 8, 64, 3500, (4, 4, "few")),
    ([17000], [9], 4, 1, 128, 10000, (4, 4, "many")),
    ([70, 20000], [1, 1], 16, 1, 64, 10000, (4, 4, "many")),
    ([100, 64, 700, 1] * 20, [5] * 80, 16, 4, 64, 40, (4, 4, "one")),
    ([10] * 300 + [17000], [1] * 301, 12, 1, 64, 280, (4, 4, "one")),
]


def _form_of(case):
    lens, new, hq, hkv, d, wide, _ = case
    rt, waves, splits = form(len(lens), sum(new), hq, hkv, d, wide)
    return rt, waves, "one" if splits == 1 else "few" if splits <= FEW else "many"


def test_forms():
    for case in CASES:
        assert _form_of(case) == case[-1], case[:1]
    # everything that the rule can give is there; 16 rows run 4 waves, and 4 waves of fewer rows are not split as far
    assert {c[-1] for c in CASES} == {(1, 16, "one"), (1, 16, "few"), (1, 16, "many"), (1, 4, "one"), (1, 4, "few"), (2, 8, "one"),
                                      (2, 8, "few"), (2, 8, "many"), (2, 4, "one"), (4, 4, "one"), (4, 4, "few"), (4, 4, "many")}
    for c in CASES:  # results of several workgroups do meet, of more than FEW of them in the other kernel
        rt, waves, splits = form(len(c[0]), sum(c[1]), *c[2:6])
        most = max(parts(up(a + b, 64), splits, waves) for a, b in zip(c[0], c[1]))
        assert most == 1 if c[-1][2] == "one" else 1 < most <= FEW if c[-1][2] == "few" else most > FEW, c[:1]
    # and a wave with a second round of pages, for each number of rows
    rounds = {(rt, waves) for c in CASES for rt, waves, splits in [form(len(c[0]), sum(c[1]), *c[2:6])]
              if max(up(up(a + b, 64), parts(up(a + b, 64), splits, waves)) for a, b in zip(c[0], c[1])) > 64 * waves}
    assert rounds >= {(1, 4), (2, 8), (2, 4), (4, 4)}


def test_rule_against_the_workspace():
    """The splits of the mirrored rule are those that the library asks workspace for."""
    import bit_ternary_weight_bitlinear_amd as lib
    if not os.path.exists(lib.library_path()):
        pytest.skip("the library is not built")
    rng = np.random.default_rng(5)
    seen = set()
    for _ in range(4000):
        seqs, d = int(np.exp(rng.uniform(0, 6.5))), int(rng.choice([64, 128]))
        hq, hkv = [(20, 5), (32, 8), (8, 8), (16, 2), (12, 4), (7, 1), (6, 2), (64, 1)][rng.integers(8)]
        m, wide = seqs * int(rng.integers(1, 12)), int(np.exp(rng.uniform(0, 9)))
        rt, waves, splits = form(seqs, m, hq, hkv, d, wide)
        need = up(splits * m * hq * d * 4, 256) * 256 + up(splits * m * hq * 8, 256) * 256 if splits > 1 else 0
        assert lib.attention_cached_workspace_size(m, hq, hkv, d, seqs, wide) == need, (seqs, m, hq, hkv, d, wide)
        seen.add((rt, waves, min(splits, FEW + 1)))
    assert len(seen) > 30


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("n", range(len(CASES)), ids=[f"{c[-1][0] * 4}rows-{c[-1][1]}waves-{c[-1][2]}-{i}" for i, c in enumerate(CASES)])
def test_every_form_against_the_definition(bl, n, weighted, dtype):  # noqa: F811
    """Long sequences take their blocks from a few pages in no order; some blocks have no page, among them ones beside
    the ends of a round of 64 pages per wave, and the row of a whole sequence's last block."""
    lens, new, hq, hkv, d, wide, (_, waves, _) = CASES[n]
    c = _Paged(bl, [640], [1], hkv, d, 31)
    rng = np.random.default_rng(n)
    c.wide, c.table = wide, rng.integers(0, c.pages, (len(lens), wide))
    for s, (a, b) in enumerate(zip(lens, new)):
        blocks = up(a + b, 64)
        c.table[s, blocks:] = -1
        if blocks > 6:
            c.table[s, [1, blocks // 2]] = -1, c.pages + 3
        for block in (64 * waves - 1, 64 * waves, 64 * waves + 1):
            if block < blocks - 1 and block % 2 == 0:
                c.table[s, block] = -1
    m = sum(new)
    q = _rand((m, hq, d), 5 + n, DTYPES[dtype], 1.5)
    first = torch.rand((len(lens), wide), generator=torch.Generator().manual_seed(n)).cuda()
    host_cu = np.concatenate([[0], np.cumsum(new)])
    want, add, spread, reach, grain = ref.attention_cached(_np(q), c.kc, c.ks, c.vc, c.vs, c.table, lens, host_cu, d ** -0.5)
    # q to 2^-22 of its row's largest (reach counts that), p to 2^-23 of its block's; a rescale per block rounds once
    r = 32 * 2.0**-24 * reach + (max(up(a + b, 64) for a, b in zip(lens, new)) + 96) * 2.0**-24
    tol = 2 * r * spread + 2.0**-22 * grain + 2.0**-24 * np.abs(want) + 1e-30 + (2.0**-8 * np.abs(want) if dtype == "bf16" else 0)
    for cu in (_starts(new), None) if all(x == 1 for x in new) else (_starts(new),):
        w = first.clone() if weighted else None
        out = bl.attention_cached(q, c.cache, _i32(c.table), _i32(lens), cu, weights=w)
        _assert_within(_np(out).reshape(m, hq, d), want, tol, f"{lens[:4]} {new[:4]}")
        if weighted:
            total = add + first.cpu().numpy()
            _assert_within(w.cpu().numpy(), total, (2 * float(r.max()) + (m * hq + 4) * 2.0**-24) * total + 1e-30, "weights")
