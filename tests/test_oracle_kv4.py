"""Pins of the 4-bit cache's oracle: the layout is a bijection, the quantiser's hand-worked values and its error
bound, the rotation's invariants, and the attention reference against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

from kv_util import attend64, block_table, build_cache4, kv4, oracle, rope_table


@pytest.mark.parametrize("d", [64, 128, 256])
def test_layout_is_a_bijection(d):
    nib = [f(d, r, x) for f in (kv4.k_nibble, kv4.v_nibble) for r in range(32) for x in range(d)]
    assert sorted(nib) == list(range(64 * d))
    # K's codes fill the first 16 d bytes, V's the next 16 d
    assert max(kv4.k_nibble(d, r, x) for r in range(32) for x in range(d)) == 32 * d - 1


def test_layout_by_hand():
    # d = 128: key 3's dims 40..47 (block 1, t = 1) are word (3 * 4 + 1) * 4 + 1 = 53
    assert kv4.k_nibble(128, 3, 40) == 8 * 53 and kv4.k_nibble(128, 3, 47) == 8 * 53 + 7
    # key 13's dim 70 (block 2, g = 1, n = 2): word ((1 * 8 + 1) * 4 + 2) * 4 + 2 = 154, the odd key's half
    assert kv4.v_nibble(128, 13, 70) == 32 * 128 + 8 * 154 + 4 + 2
    # d = 256: the second run of 128 dims follows all keys' first run
    assert kv4.k_nibble(256, 0, 128) == 8 * (32 * 16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantise_by_hand(dtype):
    x = torch.arange(32, dtype=torch.float32).to(dtype)[None]  # 0..31: scale 31 / 15
    codes, pairs = kv4.quantise(x, 32)
    s = float(torch.tensor(31 / 15).to(dtype))
    assert pairs[0, 0].tolist() == [s, 0.0]
    assert codes[0].tolist() == [min(15, round(i / s)) for i in range(32)]
    # ties go to the even code: scale 1, values at the half points
    y = torch.cat([torch.tensor([0.0, 15.0]), torch.arange(30) / 2 + 0.0]).to(dtype)[None]
    assert kv4.quantise(y, 32)[0][0, 2:].tolist() == [int(np.rint(i / 2)) for i in range(30)]
    # a constant group has scale 0, codes 0 and its own value
    c, p = kv4.quantise(torch.full((1, 32), -3.5, dtype=dtype), 32)
    assert not c.any() and kv4.values(c, p, 32).tolist() == [[-3.5] * 32]


@pytest.mark.parametrize("dtype,half", [(torch.bfloat16, 2.0 ** -8), (torch.float16, 2.0 ** -11)])
def test_quantise_error_bound(dtype, half):
    """Off by at most half a step, or, above the last level, by what the rounded scale leaves out."""
    x = (torch.from_numpy(np.random.default_rng(5).standard_normal((50, 128))) * 3 - 1).to(dtype)
    codes, pairs = kv4.quantise(x, 64)
    err = abs(kv4.values(codes, pairs, 64) - x.double().numpy())
    s = np.repeat(pairs[..., 0].double().numpy(), 64, -1)
    assert np.all(err <= s * (0.5 + 15 * half) + 1e-12)
    assert err.max() > 0.4 * s.min()


def test_write_then_read():
    rng = np.random.default_rng(0)
    for d, group in ((64, 32), (128, 128), (256, 64)):
        page = np.full(2 * kv4.unit_bytes(d, group), 0xFF, np.uint8)
        x = [torch.from_numpy(rng.standard_normal((20, d))).to(torch.bfloat16) for _ in range(2)]
        kv = tuple(kv4.quantise(t, group) for t in x)
        kv4.write(page, 25, kv, group)  # across the units' border
        for (c, p), (c2, p2) in zip(kv, kv4.read(page, 25, 20, d, group, torch.bfloat16)):
            assert np.array_equal(c, c2) and torch.equal(p, p2)
        assert int((page == 0xFF).sum()) >= page.size * 40 // 64  # the other rows keep their bytes


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_pins(interleaved):
    rng = np.random.default_rng(1)
    cs = rope_table(64, 32)
    x, y = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    r = lambda v, p: kv4.rotate(v, cs, np.array([p]), interleaved)[0]  # noqa: E731
    assert np.array_equal(r(x, 0), x)                                   # position 0 turns nothing
    assert np.array_equal(r(x, 9)[..., 32:], x[..., 32:])               # dims past the rotary width
    assert abs(np.linalg.norm(r(x, 9)) - np.linalg.norm(x)) < 1e-6
    # the product of two rows depends on the distance of their positions only
    assert abs((r(x, 30) * r(y, 23)).sum() - (r(x, 12) * r(y, 5)).sum()) < 1e-5
    assert abs((r(x, 30) * r(y, 23)).sum() - (r(x, 12) * r(y, 6)).sum()) > 1e-3
    # one quarter turn by hand: (x, y) -> (-y, x)
    quarter = np.array([[0.0, 1.0]], np.float32)
    z = kv4.rotate(np.array([[[2.0, 3.0, 7.0]]]), quarter, np.array([0]), interleaved)[0]
    assert z.tolist() == [[[-3.0, 2.0, 7.0]]]


def test_attention_reference_against_the_oracle():
    rng = np.random.default_rng(2)
    lens, hkv, g, d, group, sq = [70, 3], 2, 2, 64, 32, 3
    ks, vs = ([torch.from_numpy(rng.standard_normal((n, hkv, d))).to(torch.bfloat16) for n in lens] for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((2, sq, hkv * g, d))).to(torch.bfloat16)
    table, count = block_table(lens, 64, 0)
    cache, held = build_cache4(ks, vs, table, count, 64, group)
    for window, cap in ((-1, 0.0), (5, 4.0)):
        o, lse, o_tol, l_tol = attend64(q, held, group, 1 / math.sqrt(d), window, cap)
        for i in range(2):
            k, v = (kv4.values(*held[i][w], group)[None] for w in (0, 1))
            ro, rl = oracle.attention(q[i:i + 1].double().numpy(), k, v, causal=True, window=(window, -1), softcap=cap)
            ro = ro.reshape(hkv * g, sq, d).transpose(1, 0, 2)
            assert abs(o[i] - ro).max() < 1e-12 and abs(lse[i] - rl.reshape(hkv * g, sq)).max() < 1e-12
        assert o_tol.max() < 0.02 and l_tol.max() < 1e-3
    # what the pages hold is what was written
    for i, n in enumerate(lens):
        for p in range(math.ceil(n / 64)):
            m = min(64, n - 64 * p)
            got = kv4.read(cache[int(table[i, p]), 1], 0, m, d, group, torch.bfloat16)
            for w in (0, 1):
                assert np.array_equal(got[w][0], held[i][w][0][64 * p:64 * p + m, 1])


def test_bounds_catch_planted_mistakes():
    """A dropped min, a swapped V key pair and a shifted diagonal lie far outside the bounds."""
    rng = np.random.default_rng(3)
    n, d, group = 40, 64, 64
    k, v = (torch.from_numpy(rng.standard_normal((n, 1, d)) + 0.5).to(torch.bfloat16) for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((1, 1, 1, d))).to(torch.bfloat16)
    kq, vq = kv4.quantise(k, group), kv4.quantise(v, group)
    o, lse, o_tol, l_tol = attend64(q, [(kq, vq)], group, 0.125)
    zero = torch.cat([vq[1][..., :1], torch.zeros_like(vq[1][..., 1:])], -1)
    swap = np.arange(n) ^ 1
    for bad in ((kq, (vq[0], zero)), (kq, (vq[0][swap], vq[1][swap])),
                tuple((c[:-1], p[:-1]) for c, p in (kq, vq))):
        o2 = attend64(q, [bad], group, 0.125)[0]
        assert (abs(o2 - o) > o_tol).any()
