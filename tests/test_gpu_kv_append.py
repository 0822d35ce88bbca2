"""GPU parity of fa_kv_append, fa_kv_append_int4 and fa_kv_gather_int4 against the formulas in 64 bits.

Rotated values: each product and the sum are rounded once in fp32 (2^-24 of the products' magnitudes each, twice over
for product and sum), then once to 16 bits.  Everything that is not rotated is a copy, bit for bit.  The 4-bit codes
and pairs are those of the rows as rounded to 16 bits, bit for bit; read back they are rounded to 16 bits once more
(and once in fp32, 2^-24).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect this module
    pytest.skip("needs a GPU", allow_module_level=True)

from kv_util import DT, HALF_STEP, TINY, block_table, kv4, place, rope_table  # noqa: E402
from tiled_exact_attention_gb300 import (fa_kv_append, fa_kv_append_int4, fa_kv_gather_int4,  # noqa: E402
                                         fa_sync_status)
from tiled_exact_attention_gb300.inputs import normal  # noqa: E402

DEV = "cuda:0"

# name: new tokens and earlier keys per sequence, hq, hkv, d, dtype, page size, rotary width, interleaved, group
CASES = {
    "step": ([1, 1, 1], [0, 63, 700], 8, 2, 128, "bf16", 64, 128, False, 128),
    "step-fp16-d64": ([1] * 5, [5, 64, 127, 31, 32], 4, 4, 64, "fp16", 64, 64, True, 32),
    "prompt": ([150, 1, 64, 0, 33], [0, 64, 0, 9, 31], 8, 2, 128, "bf16", 64, 128, False, 64),
    "prompt-pairs": ([97, 130], [3, 0], 6, 2, 128, "fp16", 128, 64, True, 32),
    "partial-halves": ([45, 20], [0, 100], 5, 1, 64, "bf16", 64, 32, False, 64),
    "wide": ([70, 3], [61, 190], 3, 3, 256, "fp16", 192, 256, False, 128),
    "wide-16": ([33], [31], 2, 1, 256, "bf16", 64, 16, False, 32),
    "no-rotation": ([40, 2], [0, 5], 2, 2, 64, "bf16", 64, 0, False, 32),
    "no-queries": ([17, 50], [1, 0], 0, 2, 128, "bf16", 64, 128, True, 128),
}


def _inputs(case, seed=7):
    new, old, hq, hkv, d, dt, ps, rot, inter, group = case
    dtype, total = DT[dt], sum(new)
    lens = [a + b for a, b in zip(new, old)]
    table, count = block_table(lens, ps, seed)
    x = {n: normal((total, h, d), seed, i, 1.5, dtype) for i, (n, h) in enumerate((("q", max(hq, 1)), ("k", hkv), ("v", hkv)))}
    cs = rope_table(max(lens) + 1, rot) if rot else None
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return x, cs, cu, lens, table, count


def _dev(a):
    return None if a is None else torch.from_numpy(a).to(DEV)


def _expected(case, x, cs, lens, name):
    """Rows in 64 bits and their bound."""
    new, _, _, _, _, dt, _, rot, inter, _ = case
    v = x[name].double().numpy()
    if not rot:
        return v, np.zeros_like(v)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)]) if sum(new) else np.zeros(0, int)
    y, size = kv4.rotate(v, cs, pos, inter)
    fp32 = 2 * 2.0 ** -24 * size * 1.001
    u = HALF_STEP[DT[dt]]
    tol = np.where(size > 0, u * (abs(y) + fp32) + fp32 + TINY[DT[dt]], 0.0)
    return y, tol


def _kw(case, x, cs, cu, lens, table, **more):
    hq = case[2]
    return dict(block_table=_dev(table), seqlens_k=torch.tensor(lens, dtype=torch.int32, device=DEV),
                cu_seqlens=_dev(cu), q=x["q"].to(DEV) if hq else None, cos_sin=_dev(cs), interleaved=case[8], **more)


def _within(got, ref, tol, what):
    d = abs(got.double().cpu().numpy() - ref)
    assert (d <= tol).all(), f"{what}: off by {d.max():.3e}"


@pytest.mark.parametrize("name", CASES)
def test_append(name):
    case = CASES[name]
    new, old, hq, hkv, d, dt, ps, rot, inter, _ = case
    x, cs, cu, lens, table, count = _inputs(case)
    kc, vc = (normal((count, ps, hkv, d), 3, i, 1.0, DT[dt]) for i in (0, 1))
    kg, vg = kc.to(DEV), vc.to(DEV)
    q = fa_kv_append(x["k"].to(DEV), x["v"].to(DEV), kg, vg, **_kw(case, x, cs, cu, lens, table))
    assert fa_sync_status() == 0
    ek, tk = _expected(case, x, cs, lens, "k")
    rk, rt = kc.double().numpy(), np.zeros(kc.shape)
    for i, n in enumerate(new):
        for t in range(n):
            at = place(table, ps, i, lens[i] - n + t)
            rk[at], rt[at] = ek[cu[i] + t], tk[cu[i] + t]
            vc[at] = x["v"][cu[i] + t]
    _within(kg, rk, rt, "K cache")  # untouched rows exactly
    assert torch.equal(vg.cpu(), vc)
    if hq:
        _within(q, *_expected(case, x, cs, lens, "q"), "q")
    else:
        assert q is None


@pytest.mark.parametrize("name", CASES)
def test_append_int4_and_gather(name):
    case = CASES[name]
    new, old, hq, hkv, d, dt, ps, rot, inter, group = case
    x, cs, cu, lens, table, count = _inputs(case)
    dtype = DT[dt]
    before = np.random.default_rng(1).integers(0, 256, (count, hkv, ps // 32 * kv4.unit_bytes(d, group))).astype(np.uint8)
    cache = _dev(before)
    kw = _kw(case, x, cs, cu, lens, table)
    q = fa_kv_append_int4(x["k"].to(DEV), x["v"].to(DEV), cache, group=group, **kw)
    # the 16-bit append gives the rows that are quantised
    k16, v16 = (torch.zeros((count, ps, hkv, d), dtype=dtype, device=DEV) for _ in range(2))
    q16 = fa_kv_append(x["k"].to(DEV), x["v"].to(DEV), k16, v16, **kw)
    assert fa_sync_status() == 0
    assert q is None if not hq else torch.equal(q, q16)
    k16 = k16.cpu()
    want = before.copy()
    rows = {"k": torch.zeros_like(x["k"]), "v": x["v"]}
    for i, n in enumerate(new):
        for t in range(n):
            rows["k"][cu[i] + t] = k16[place(table, ps, i, lens[i] - n + t)]
    kq, vq = (kv4.quantise(rows[n], group) for n in ("k", "v"))
    for i, n in enumerate(new):
        for t in range(n):
            r = slice(cu[i] + t, cu[i] + t + 1)
            page, row = place(table, ps, i, lens[i] - n + t)
            for h in range(hkv):
                kv4.write(want[page, h], row, tuple((c[r, h], p[r, h]) for c, p in (kq, vq)), group)
    assert np.array_equal(cache.cpu().numpy(), want)
    kb, vb = fa_kv_gather_int4(cache, group=group, block_table=kw["block_table"], seqlens_k=kw["seqlens_k"],
                               cu_seqlens=kw["cu_seqlens"], total=sum(new), d=d, dtype=dtype)
    assert fa_sync_status() == 0
    for got, (c, p) in ((kb, kq), (vb, vq)):
        ref = kv4.values(c, p, group)
        mag = abs(ref) + 2.0 ** -24 * (abs(ref) + 1e-30)
        _within(got, ref, HALF_STEP[dtype] * mag + 2.0 ** -24 * abs(ref) + TINY[dtype], "gather")


def test_prefixes_and_whole_sequences():
    """Gathering whole sequences with other lengths than the append's, rows of no sequence left alone."""
    case = CASES["prompt"]
    x, cs, cu, lens, table, count = _inputs(case)
    new, group, d, hkv = case[0], 64, 128, 2
    cache = torch.zeros((count, hkv, 64 // 32 * kv4.unit_bytes(d, group)), dtype=torch.uint8, device=DEV)
    kw = _kw(case, x, cs, cu, lens, table)
    fa_kv_append_int4(x["k"].to(DEV), x["v"].to(DEV), cache, group=group, **kw)
    full = np.concatenate([[4], 4 + np.cumsum(lens)]).astype(np.int32)
    k = torch.full((int(full[-1]) + 7, hkv, d), 9.0, dtype=torch.bfloat16, device=DEV)
    v = torch.full_like(k, 8.0)
    fa_kv_gather_int4(cache, group=group, block_table=kw["block_table"], seqlens_k=kw["seqlens_k"],
                      cu_seqlens=_dev(full), k_out=k, v_out=v)
    kb, vb = fa_kv_gather_int4(cache, group=group, block_table=kw["block_table"], seqlens_k=kw["seqlens_k"],
                               cu_seqlens=kw["cu_seqlens"], total=sum(new), d=d, dtype=torch.bfloat16)
    assert fa_sync_status() == 0
    for i, n in enumerate(new):
        assert torch.equal(k[full[i + 1] - n:full[i + 1]], kb[cu[i]:cu[i + 1]])
        assert torch.equal(v[full[i + 1] - n:full[i + 1]], vb[cu[i]:cu[i + 1]])
    assert (k[:4] == 9).all() and (k[full[-1]:] == 9).all() and (v[:4] == 8).all() and (v[full[-1]:] == 8).all()


@pytest.mark.parametrize("int4", [False, True])
def test_views_in_place_and_uniform(int4):
    """q, k and v as views of one projection, q_out = q, every sequence the same number of tokens."""
    b, n, hq, hkv, d, ps = 3, 5, 4, 2, 128, 64
    lens = [5, 70, 128]
    table, count = block_table(lens, ps, 2, width=4)
    qkv = normal((b * n, hq + 2 * hkv, d), 5, 0, 1.0, torch.bfloat16)
    cs = rope_table(200, 128)
    cu = _dev(np.arange(0, b * n + 1, n, dtype=np.int32))
    wide = torch.zeros((b, 9), dtype=torch.int32, device=DEV)
    wide[:, :4] = _dev(table)

    def go(g, q_out, **kw):
        q, k, v = g[:, :hq], g[:, hq:hq + hkv], g[:, hq + hkv:]
        kw = dict(q=q, q_out=q if q_out is None else q_out, cos_sin=_dev(cs), interleaved=True,
                  seqlens_k=torch.tensor(lens, dtype=torch.int32, device=DEV), **kw)
        if int4:
            c = torch.zeros((count, hkv, 2 * kv4.unit_bytes(d, 32)), dtype=torch.uint8, device=DEV)
            return fa_kv_append_int4(k, v, c, group=32, **kw), c
        # caches with the heads outside the rows
        c = torch.zeros((2, count, hkv, ps, d), dtype=torch.bfloat16, device=DEV)
        return fa_kv_append(k, v, c[0].transpose(1, 2), c[1].transpose(1, 2), **kw), c

    a, ca = go(qkv.to(DEV), torch.empty((b * n, hq, d), dtype=torch.bfloat16, device=DEV), block_table=_dev(table),
               cu_seqlens=cu)
    g = qkv.to(DEV)
    e, ce = go(g, None, block_table=wide[:, :4])  # in place; a table with rows apart
    assert fa_sync_status() == 0
    assert torch.equal(a, e) and torch.equal(ca, ce) and e.data_ptr() == g.data_ptr()
    assert torch.equal(g[:, hq:].cpu(), qkv[:, hq:])


@pytest.mark.parametrize("int4", [False, True])
def test_padding_tokens_and_rows_of_no_sequence(int4):
    """Tokens at negative positions and rows outside the prefix sums: nothing is written, q_out keeps its rows."""
    hkv, d, ps = 1, 64, 64
    k = normal((20, hkv, d), 1, 0, 1.0, torch.float16).to(DEV)
    q_out = torch.full((20, 2, d), 5.0, dtype=torch.float16, device=DEV)
    q = normal((20, 2, d), 1, 1, 1.0, torch.float16).to(DEV)
    cs = _dev(rope_table(10, 64))
    kw = dict(block_table=torch.tensor([[0], [1], [2]], dtype=torch.int32, device=DEV),
              seqlens_k=torch.tensor([0, 3, 2], dtype=torch.int32, device=DEV),
              cu_seqlens=torch.tensor([2, 4, 9, 11], dtype=torch.int32, device=DEV), q=q, q_out=q_out, cos_sin=cs)
    shape = (4, hkv, 2 * kv4.unit_bytes(d, 64)) if int4 else (4, ps, hkv, d)
    c = torch.full(shape, 7, dtype=torch.uint8 if int4 else torch.float16, device=DEV)
    if int4:
        fa_kv_append_int4(k, k, c, group=64, **kw)
    else:
        fa_kv_append(k, k, c, c.clone(), **kw)
    assert fa_sync_status() == 0
    written = [i for i in range(20) if not (q_out[i] == 5).all()]
    assert written == [6, 7, 8, 9, 10]  # three of the second sequence's five tokens, both of the third
    assert (c[0] == 7).all() and (c[3] == 7).all() and not (c[1] == 7).all()


BAD = {
    "page out of range": dict(table=[[0], [64]], lens=[3, 3], cu=[0, 3, 6]),
    "page negative": dict(table=[[0], [-1]], lens=[3, 3], cu=[0, 3, 6]),
    "past the table": dict(table=[[0], [1]], lens=[3, 66], cu=[0, 3, 6]),
    "past the rotation table": dict(table=[[0], [1]], lens=[3, 51], cu=[0, 3, 6]),
    "decreasing prefix sums": dict(table=[[0], [1]], lens=[3, 3], cu=[0, 3, 1]),
    "prefix sums past the rows": dict(table=[[0], [1]], lens=[3, 5], cu=[0, 3, 8]),
    "negative prefix sum": dict(table=[[0], [1]], lens=[3, 3], cu=[-2, 3, 6]),
}


@pytest.mark.parametrize("name,op", [(n, o) for n in BAD for o in ("append", "append4", "gather")
                                     if o != "gather" or "rotation" not in n])
def test_device_side_refusals(name, op):
    """A bad argument read on the device is reported; the other sequence is served and nothing else is written."""
    bad, hkv, d = BAD[name], 1, 64
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    kw = dict(block_table=ints(bad["table"]), seqlens_k=ints(bad["lens"]), cu_seqlens=ints(bad["cu"]))
    k = normal((6, hkv, d), 1, 0, 1.0, torch.bfloat16).to(DEV)
    cs = _dev(rope_table(50, 64))
    if op == "append":
        c = torch.full((4, 64, hkv, d), 7.0, dtype=torch.bfloat16, device=DEV)
        fa_kv_append(k, k, c, torch.zeros_like(c), cos_sin=cs, **kw)
        assert fa_sync_status() == 6
        assert (c[2:] == 7).all()
        assert bad["cu"][0] < 0 or (c[0, :3] != 7).any()
    elif op == "append4":
        c = torch.full((4, hkv, 2 * kv4.unit_bytes(d, 32)), 7, dtype=torch.uint8, device=DEV)
        fa_kv_append_int4(k, k, c, group=32, cos_sin=cs, **kw)
        assert fa_sync_status() == 6
        assert (c[2:] == 7).all()
    else:
        c = torch.zeros((4, hkv, 2 * kv4.unit_bytes(d, 32)), dtype=torch.uint8, device=DEV)
        fa_kv_gather_int4(c, group=32, k_out=k, v_out=k.clone(), **kw)
        assert fa_sync_status() == 6
    assert fa_sync_status() == 0


def test_wrapper_refusals():
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    c = torch.zeros(2, 64, 2, 64, dtype=torch.bfloat16, device=DEV)
    c4 = torch.zeros(2, 2, 64 * 72, dtype=torch.uint8, device=DEV)
    t, n = torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    ok = dict(block_table=t, seqlens_k=n)
    cs = torch.zeros(8, 64, device=DEV)
    for call in (
        lambda: fa_kv_append(k, k[:, :1], c, c, **ok),
        lambda: fa_kv_append(k, k.half(), c, c, **ok),
        lambda: fa_kv_append(k, k, c[..., :32], c, **ok),
        lambda: fa_kv_append(k, k, c, c, block_table=t.long(), seqlens_k=n),
        lambda: fa_kv_append(k, k, c, c, block_table=t, seqlens_k=n[:1]),
        lambda: fa_kv_append(k, k, c, c, cu_seqlens=n, **ok),
        lambda: fa_kv_append(k[:3], k[:3], c, c, **ok),
        lambda: fa_kv_append(k, k, c, c, cos_sin=cs.half(), **ok),
        lambda: fa_kv_append(k, k, c, c, cos_sin=cs, rotary_dim=32, **ok),
        lambda: fa_kv_append(k, k, c, c, rotary_dim=32, **ok),
        lambda: fa_kv_append(k, k, c, c, q_out=k, **ok),
        lambda: fa_kv_append(k, k, c, c, q=k[:2], **ok),
        lambda: fa_kv_append(k, k, c, c, q=k.transpose(1, 2), **ok),
        lambda: fa_kv_append_int4(k, k, c4, group=48, **ok),
        lambda: fa_kv_append_int4(k, k, c4, group=128, **ok),
        lambda: fa_kv_append_int4(k, k, c4, group=32, **ok),
        lambda: fa_kv_append_int4(k, k, c4[:, :1], group=64, **ok),
        lambda: fa_kv_gather_int4(c4, group=64, k_out=k, **ok),
        lambda: fa_kv_gather_int4(c4, group=64, k_out=k, v_out=k[:, :1], **ok),
    ):
        with pytest.raises(ValueError):
            call()
    assert fa_sync_status() == 0


@pytest.mark.parametrize("int4", [False, True])
def test_other_stream_and_graph(int4):
    """On an explicit stream, and captured: replays read the lengths and inputs that the tensors then hold."""
    b, hq, hkv, d, ps = 4, 4, 2, 128, 64
    table, count = block_table([200] * b, ps, 4)
    table = _dev(table)
    lens = torch.tensor([1, 60, 64, 129], dtype=torch.int32, device=DEV)
    cs = _dev(rope_table(256, 128))
    x = [normal((b, h, d), 9, i, 1.0, torch.bfloat16).to(DEV) for i, h in enumerate((hq, hkv, hkv))]
    shape = (count, hkv, 2 * kv4.unit_bytes(d, 128)) if int4 else (2, count, ps, hkv, d)

    def step(c, q, k, v, lens, **kw):
        kw.update(block_table=table, seqlens_k=lens, q=q, cos_sin=cs)
        if int4:
            return fa_kv_append_int4(k, v, c, group=128, **kw)
        return fa_kv_append(k, v, c[0], c[1], **kw)

    new = lambda: torch.zeros(shape, dtype=torch.uint8 if int4 else torch.bfloat16, device=DEV)  # noqa: E731
    want, side, graphed = new(), new(), new()
    q0 = step(want, *x, lens)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    q1 = step(side, *x, lens, stream=st)
    st.synchronize()
    assert torch.equal(q0, q1) and torch.equal(want, side)
    static = [t.clone() for t in x] + [lens.clone()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q2 = step(graphed, *static)
    for add in (0, 1, 37):
        l2 = lens + add
        y = [t * (1 + add) for t in x]
        for dst, src in zip(static, y + [l2]):
            dst.copy_(src)
        g.replay()
        q3 = step(want, *y, l2)
        torch.cuda.synchronize()
        assert torch.equal(q2, q3) and torch.equal(want, graphed)
    assert fa_sync_status() == 0
