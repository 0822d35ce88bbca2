"""GPU parity of fa_fwd_kvcache_int4 (attention of a few query tokens over a 4-bit paged cache) against the definition
in 64 bits on the held values; the bounds are derived in kv_util.attend64.  Bytes of the cache that no key owns are
0xFF (NaN pairs), table entries that no key reaches are out of range."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect this module
    pytest.skip("needs a GPU", allow_module_level=True)

from kv_util import DT, attend64, block_table, build_cache4, check_attention, kv4, rope_table  # noqa: E402
from tiled_exact_attention_gb300 import (fa_fwd_kvcache, fa_fwd_kvcache_int4, fa_fwd_varlen, fa_kv_append,  # noqa: E402
                                         fa_kv_append_int4, fa_kv_gather_int4, fa_sync_status)
from tiled_exact_attention_gb300.inputs import normal  # noqa: E402

DEV = "cuda:0"


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _rows(lens, hkv, d, dt, seed, std=1.0):
    return [[normal((n, hkv, d), seed, 10 + 2 * i + w, std, dt) for i, n in enumerate(lens)] for w in (0, 1)]


# name: lengths, sq, hq, hkv, d, group, dtype, page size, window, softcap
CASES = {
    "one-key": ([1], 1, 4, 1, 128, 128, "bf16", 64, -1, 0.0),
    "edges": ([1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129], 1, 4, 2, 128, 128, "bf16", 64, -1, 0.0),
    "empty": ([0, 5, 0], 1, 8, 2, 64, 64, "fp16", 64, -1, 0.0),
    "long": ([3001, 64, 900], 1, 8, 2, 128, 64, "bf16", 128, -1, 0.0),
    "fine": ([777, 2050], 1, 8, 2, 128, 32, "fp16", 192, -1, 0.0),
    "one-head-each": ([500, 33], 1, 3, 3, 64, 32, "bf16", 64, -1, 0.0),
    "wide": ([260, 1025], 1, 4, 2, 256, 128, "bf16", 64, -1, 0.0),
    "wide-fine": ([300, 40], 1, 4, 2, 256, 32, "fp16", 64, -1, 0.0),
    "wide-64": ([100, 640], 1, 2, 1, 256, 64, "fp16", 64, -1, 0.0),
    "nine-heads": ([130, 400], 1, 18, 2, 128, 128, "fp16", 64, -1, 0.0),
    "many-heads": ([70, 333], 1, 40, 1, 64, 64, "bf16", 64, -1, 0.0),
    "drafted": ([3, 4, 5, 200, 1], 4, 8, 2, 128, 128, "bf16", 64, -1, 0.0),
    "drafted-wide-group": ([65, 300], 7, 10, 2, 64, 32, "fp16", 64, -1, 0.0),
    "drafted-d256": ([90, 20], 3, 16, 2, 256, 64, "bf16", 64, -1, 0.0),
    "window": ([1000, 10, 64], 1, 4, 2, 128, 64, "bf16", 64, 100, 0.0),
    "window-all": ([300, 1], 2, 4, 2, 128, 64, "bf16", 64, (1 << 31) - 1, 0.0),
    "window-0": ([130, 1], 1, 4, 2, 64, 64, "fp16", 64, 0, 0.0),
    "window-drafted": ([700, 33, 2], 5, 8, 2, 128, 128, "fp16", 64, 37, 0.0),
    "softcap": ([500, 70], 1, 8, 2, 128, 128, "bf16", 64, -1, 5.0),
    "all": ([1500, 129, 3], 3, 12, 2, 128, 32, "bf16", 128, 300, 20.0),
}


def _problem(case, seed=11, k_std=1.0):
    lens, sq, hq, hkv, d, group, dt, ps, window, cap = case
    dtype = DT[dt]
    ks, vs = _rows(lens, hkv, d, dtype, seed, k_std)
    q = normal((len(lens), sq, hq, d), seed, 1, 1.0, dtype)
    table, count = block_table(lens, ps, seed)
    cache, held = build_cache4(ks, vs, table, count, ps, group)
    return q, cache, held, table


def _run(case, q, cache, table, **kw):
    lens, sq, hq, hkv, d, group, dt, ps, window, cap = case
    return fa_fwd_kvcache_int4(q.to(DEV), torch.from_numpy(cache).to(DEV), group=group,
                               block_table=torch.from_numpy(table).to(DEV), seqlens_k=ints(lens),
                               window_left=window if window >= 0 else None, softcap=cap, **kw)


@pytest.mark.parametrize("name", CASES)
def test_parity(name):
    case = CASES[name]
    q, cache, held, table = _problem(case)
    o, lse = _run(case, q, cache, table)
    assert fa_sync_status() == 0
    ref = attend64(q, held, case[5], 1 / math.sqrt(case[4]), case[8], case[9])
    check_attention(o, lse, ref, name)


def _fuzz(n=24):
    rng = np.random.default_rng(2026)
    for i in range(n):
        d = int(rng.choice([64, 128, 256]))
        hkv, g, sq = int(rng.integers(1, 4)), int(rng.choice([1, 2, 3, 4, 5, 8])), int(rng.choice([1, 1, 2, 3, 6]))
        lens = [int(x) for x in rng.integers(0, 400, int(rng.integers(1, 6)))]
        yield (lens, sq, g * hkv, hkv, d, int(rng.choice([x for x in (32, 64, 128) if x <= d])),
               str(rng.choice(["bf16", "fp16"])), int(rng.choice([64, 128, 192])),
               int(rng.choice([-1, -1, 3, 60, 250])), float(rng.choice([0.0, 0.0, 8.0])))


@pytest.mark.parametrize("i,case", list(enumerate(_fuzz())), ids=lambda x: str(x) if isinstance(x, int) else "")
def test_random_shapes(i, case):
    q, cache, held, table = _problem(case, 100 + i)
    o, lse = _run(case, q, cache, table)
    assert fa_sync_status() == 0
    check_attention(o, lse, attend64(q, held, case[5], 1 / math.sqrt(case[4]), case[8], case[9]), str(case))


def test_many_sequences_of_uneven_length():
    """More sequences than a warp has lanes, in sizes from nothing to many pages."""
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(0, 90, 100)]
    lens[17], lens[60] = 1900, 700
    case = (lens, 1, 4, 1, 64, 64, "bf16", 64, -1, 0.0)
    q, cache, held, table = _problem(case)
    o, lse = _run(case, q, cache, table)
    assert fa_sync_status() == 0
    check_attention(o, lse, attend64(q, held, 64, 0.125), "uneven")


@pytest.mark.parametrize("what", ["peaky", "large", "small", "constant", "rising-v", "sink"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_hard_values(what, dt):
    """Score ranges of hundreds, values far from 1 in size (fp16's range at both ends), groups without spread, values
    whose scales differ by orders of magnitude between keys."""
    case = ([700, 90], 1, 4, 2, 128, 64, dt, 64, -1, 0.0)
    lens, dtype = case[0], DT[dt]
    ks, vs = _rows(lens, 2, 128, dtype, 3)
    q = normal((2, 1, 4, 128), 3, 1, 1.0, dtype)
    if what == "peaky":
        ks = [(k.float() * 20).to(dtype) for k in ks]
    elif what == "large":
        top = 1e4 if dt == "fp16" else 1e30
        vs = [(v.float() * top).to(dtype) for v in vs]
    elif what == "small":
        low = 1e-4 if dt == "fp16" else 1e-25
        vs = [(v.float() * low).to(dtype) for v in vs]
        q = (q.float() * 1e-3).to(dtype)
    elif what == "constant":
        ks = [torch.full_like(k, 0.75) for k in ks]
        vs = [torch.full_like(v, -2.5) for v in vs]
    elif what == "rising-v":
        vs = [(v.float() * (2.0 ** (torch.arange(v.shape[0]) % 300 / 25))[:, None, None]).to(dtype) for v in vs]
    else:  # the first key has small values and most of the weight
        ks[0][0] = ks[0][0] * 0 + 2.0
        q = q.abs()
        vs[0][0] = vs[0][0] * 0.02
    table, count = block_table(lens, 64, 1)
    cache, held = build_cache4(ks, vs, table, count, 64, 64)
    o, lse = _run(case, q, cache, table)
    assert fa_sync_status() == 0
    check_attention(o, lse, attend64(q, held, 64, 1 / math.sqrt(128)), what)


def test_strides_outputs_and_three_dims():
    """q and out as views with the heads apart, caches with pages apart, q without the token dimension."""
    case = ([300, 65], 1, 8, 2, 128, 128, "bf16", 64, -1, 0.0)
    q, cache, held, table = _problem(case)
    o, lse = _run(case, q, cache, table)
    qg = q.to(DEV)[:, 0].transpose(0, 1).contiguous().transpose(0, 1)  # [b, hq, d], heads outermost in memory
    big = torch.full((len(cache), 2, 2, cache.shape[2]), 255, dtype=torch.uint8, device=DEV)
    big[:, 1] = torch.from_numpy(cache).to(DEV)
    wide = torch.zeros((2, 11), dtype=torch.int32, device=DEV)
    wide[:, 3:3 + table.shape[1]] = torch.from_numpy(table).to(DEV)
    out = torch.zeros((8, 2, 160), dtype=torch.bfloat16, device=DEV)[..., :128].transpose(0, 1)
    l2 = torch.zeros((2, 8), device=DEV)
    o2, l3 = fa_fwd_kvcache_int4(qg, big[:, 1], group=128, block_table=wide[:, 3:3 + table.shape[1]],
                                 seqlens_k=ints(case[0]), out=out, lse=l2)
    assert fa_sync_status() == 0
    assert o2 is out and l3 is l2
    assert torch.equal(o2, o[:, 0]) and torch.equal(l2, lse[:, :, 0])


def test_scale_and_repeatability():
    """An explicit scale; the same call twice gives the same bits."""
    case = ([2000, 1], 2, 16, 2, 64, 32, "fp16", 64, -1, 0.0)
    q, cache, held, table = _problem(case)
    o, lse = _run(case, q, cache, table, scale=0.3)
    o2, lse2 = _run(case, q, cache, table, scale=0.3)
    assert fa_sync_status() == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_attention(o, lse, attend64(q, held, 32, 0.3), "scale")


def test_bad_lengths_and_pages():
    """A sequence past its table row or with a page out of range is reported; the others are computed."""
    case = ([200, 130, 90], 1, 4, 2, 64, 64, "bf16", 64, -1, 0.0)
    q, cache, held, table = _problem(case)
    ref = attend64(q, held, 64, 0.125)
    bad = table.copy()
    bad[1, 1] = len(cache)
    for t, lens in ((table, [200, table.shape[1] * 64 + 1, 90]), (bad, [200, 130, 90]),
                    (np.where(bad == len(cache), -5, bad), [200, 130, 90])):
        o, lse = _run((lens,) + case[1:], q, cache, t.astype(np.int32))
        assert fa_sync_status() == 6
        assert fa_sync_status() == 0
        for i in (0, 2):
            check_attention(o[i:i + 1], lse[i:i + 1], tuple(r[i:i + 1] for r in ref), f"sequence {i}")
    # a negative length counts as none
    o, lse = _run(([200, -3, 90],) + case[1:], q, cache, table)
    assert fa_sync_status() == 0
    assert torch.isneginf(lse[1]).all() and (o[1] == 0).all()


def test_wrapper_refusals():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    c = torch.zeros(3, 2, 64 * 72, dtype=torch.uint8, device=DEV)
    t, n = torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    go = lambda q=q, c=c, group=64, t=t, n=n, **kw: fa_fwd_kvcache_int4(q, c, group=group, block_table=t,  # noqa: E731
                                                                       seqlens_k=n, **kw)
    go()
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(q=q[..., :32]), dict(q=q.transpose(1, 2)), dict(c=c[..., :-72]),
               dict(c=c.int()), dict(c=c[0]), dict(group=32), dict(group=128), dict(t=t.long()), dict(t=t[:1]),
               dict(n=n[:1]), dict(n=n.float()), dict(out=q[:1]), dict(out=q.half()),
               dict(lse=torch.zeros(2, 4, 1, device=DEV)), dict(lse=torch.zeros(2, 4, device=DEV).half())):
        with pytest.raises(ValueError):
            go(**kw)
    import tiled_exact_attention_gb300 as fa
    for kw in (dict(scale=0.0), dict(softcap=-1.0), dict(window_left=-2), dict(q=q[:, :3].contiguous()),
               dict(workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(fa.FaError):
            go(**kw)
    assert fa_sync_status() == 0


def test_other_stream_graph_and_two_graphs():
    """On an explicit stream, and captured with the lengths read at replay; two graphs with the same workspace, replayed
    one after the other, and an eager call between them."""
    case = ([900, 333], 1, 8, 2, 128, 128, "bf16", 64, -1, 0.0)
    q, cache, held, table = _problem(case)
    qg, cg, tg, lens = q.to(DEV), torch.from_numpy(cache).to(DEV), torch.from_numpy(table).to(DEV), ints([900, 333])
    go = lambda n, **kw: fa_fwd_kvcache_int4(qg, cg, group=128, block_table=tg, seqlens_k=n, **kw)  # noqa: E731
    want = {n: go(ints(list(n))) for n in ((900, 333), (5, 64), (640, 0))}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o, lse = go(lens, stream=st)
    st.synchronize()
    assert torch.equal(o, want[900, 333][0]) and torch.equal(lse, want[900, 333][1])
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, go(lens, workspace=ws)))
    for n in want:
        lens.copy_(ints(list(n)))
        for g, out in graphs:
            g.replay()
            eager = go(lens, workspace=ws)
            torch.cuda.synchronize()
            for x, y, z in zip(out, want[n], eager):
                assert torch.equal(x, y) and torch.equal(y, z)
    assert fa_sync_status() == 0


def test_workspace_is_free_after_the_call():
    """A call that could cut its items but cuts none leaves its workspace alone once the stream has passed it."""
    q, cache, held, table = _problem(([900, 333], 1, 8, 2, 128, 128, "bf16", 64, -1, 0.0))
    qg, cg, tg = q.to(DEV), torch.from_numpy(cache).to(DEV), torch.from_numpy(table).to(DEV)
    tg = torch.nn.functional.pad(tg, (0, 64), value=1 << 29)  # a table for much longer sequences
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    for lens in ([0, 0], [1, 3], [64, 40]):
        n = ints(lens)
        for _ in range(50):
            fa_fwd_kvcache_int4(qg, cg, group=128, block_table=tg, seqlens_k=n, workspace=ws)
            ws.fill_(0xA5)
        assert bool((ws == 0xA5).all())
    assert fa_sync_status() == 0


@pytest.mark.parametrize("dt,d,group,interleaved", [("bf16", 128, 64, False), ("fp16", 64, 32, True)])
def test_serving_run(dt, d, group, interleaved):
    """Prompts into the 4-bit cache, their attention over what the cache holds (gather + fa_fwd_varlen), a second chunk,
    then decode steps and one step of three drafted tokens; each answer against the definition on the held values."""
    dtype, hq, hkv, ps, b = DT[dt], 4, 2, 64, 3
    rng = np.random.default_rng(8)
    chunks = [[50, 1, 131], [20, 64, 3], [1, 1, 1], [1, 1, 1], [3, 3, 3], [1, 1, 1]]
    total = [sum(c[i] for c in chunks) for i in range(b)]
    table, count = block_table(total, ps, 5)
    tg = torch.from_numpy(table).to(DEV)
    cs = rope_table(max(total), d)
    cache = torch.from_numpy(np.full((count, hkv, 2 * kv4.unit_bytes(d, group)), 0xFF, np.uint8)).to(DEV)
    lens = [0] * b
    for step, new in enumerate(chunks):
        lens = [a + n for a, n in zip(lens, new)]
        cu = ints([0] + list(np.cumsum(new)))
        q, k, v = (torch.from_numpy(rng.standard_normal((sum(new), h, d))).to(dtype) for h in (hq, hkv, hkv))
        kw = dict(group=group, block_table=tg, seqlens_k=ints(lens))
        qr = fa_kv_append_int4(k.to(DEV), v.to(DEV), cache, cu_seqlens=cu, q=q.to(DEV),
                               cos_sin=torch.from_numpy(cs).to(DEV), interleaved=interleaved, **kw)
        host = cache.cpu().numpy()
        held = []
        for i, n in enumerate(lens):
            per = [[kv4.read(host[int(table[i, p]), h], 0, min(ps, n - p * ps), d, group, dtype) for h in range(hkv)]
                   for p in range(math.ceil(n / ps))]
            held.append(tuple((np.concatenate([np.stack([x[w][0] for x in row], 1) for row in per]),
                               torch.cat([torch.stack([x[w][1] for x in row], 1) for row in per])) for w in (0, 1)))
        if len(set(new)) > 1:  # a prompt's chunk
            cu_k = ints([0] + list(np.cumsum(lens)))
            kb, vb = fa_kv_gather_int4(cache, cu_seqlens=cu_k, total=sum(lens), d=d, dtype=dtype, **kw)
            o, lse = fa_fwd_varlen(qr, kb, vb, cu, cu_k, causal=True)
            for i, n in enumerate(new):
                rows = slice(sum(new[:i]), sum(new[:i + 1]))
                ref = attend64(qr[rows].cpu()[None], [held[i]], group, 1 / math.sqrt(d))
                # (the prefill rounds K, V and P to 16 bits: the framework's own tolerances)
                assert abs(o[rows].double().cpu().numpy() - ref[0][0]).max() <= (2e-2 if dt == "bf16" else 4e-3)
                assert abs(lse[:, rows].double().cpu().numpy() - ref[1][0]).max() <= (2e-2 if dt == "bf16" else 2e-3)
        else:
            o, lse = fa_fwd_kvcache_int4(qr.view(b, new[0], hq, d), cache, **kw)
            ref = attend64(qr.view(b, new[0], hq, d).cpu(), held, group, 1 / math.sqrt(d))
            check_attention(o, lse, ref, f"step {step}")
        assert fa_sync_status() == 0


def test_serving_run_16bit():
    """fa_kv_append fills what fa_fwd_kvcache reads: three steps against a dense copy of the rotated rows."""
    b, hq, hkv, d, ps = 3, 8, 2, 128, 64
    new = [[70, 5, 64], [1, 1, 1], [1, 1, 1]]
    total = [sum(c[i] for c in new) for i in range(b)]
    table, count = block_table(total, ps, 6)
    kc, vc = (torch.full((count, ps, hkv, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cs = torch.from_numpy(rope_table(200, d)).to(DEV)
    lens, dense = [0] * b, [[[], []] for _ in range(b)]
    for step, n in enumerate(new):
        lens = [a + x for a, x in zip(lens, n)]
        q, k, v = (normal((sum(n), h, d), 20 + step, i, 1.0, torch.bfloat16).to(DEV) for i, h in enumerate((hq, hkv, hkv)))
        kw = dict(block_table=torch.from_numpy(table).to(DEV), seqlens_k=ints(lens))
        qr = fa_kv_append(k, v, kc, vc, cu_seqlens=ints([0] + list(np.cumsum(n))), q=q, cos_sin=cs, **kw)
        for i in range(b):
            at = sum(n[:i])
            pos = np.arange(lens[i] - n[i], lens[i])
            kr = kv4.rotate(k[at:at + n[i]].double().cpu().numpy(), cs.cpu().numpy(), pos, False)[0]
            dense[i][0].append(torch.from_numpy(kr).to(torch.bfloat16).double().numpy())
            dense[i][1].append(v[at:at + n[i]].double().cpu().numpy())
        if step == 0:
            continue
        o, lse = fa_fwd_kvcache(qr, kc, vc, **kw)
        assert fa_sync_status() == 0
        for i in range(b):
            import oracle

            kk, vv = (np.concatenate(x)[None] for x in dense[i])
            ro, rl = oracle.attention(qr[i].double().cpu().numpy()[None, None], kk, vv, causal=False)
            assert abs(o[i].double().cpu().numpy() - ro).max() <= 1e-2
            assert abs(lse[i].double().cpu().numpy() - rl).max() <= 1e-3
