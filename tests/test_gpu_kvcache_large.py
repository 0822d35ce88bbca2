"""The paged cache's operators where offsets, lengths and tables get large or odd: caches past 4 GB, sequences past 10^5
keys, pages that hold whole sequences, one table row for all sequences, tables that are views, two calls at once; and appends
of every size in between."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect this module
    pytest.skip("needs a GPU", allow_module_level=True)

from tiled_exact_attention_gb300 import (fa_fwd_kvcache_int4, fa_kv_append, fa_kv_append_int4,  # noqa: E402
                                         fa_kv_gather_int4, fa_kvcache_int4_page_bytes, fa_sync_status)

DEV = "cuda:0"


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _exact_rows(n, h, d, group, dtype, gen):
    """Rows that a 4-bit cache holds exactly: multiples of 1/4 from -2 to 7/4 with both ends in every group."""
    x = torch.randint(0, 16, (n, h, d), generator=gen, device=DEV)
    x[..., ::group], x[..., group - 1::group] = 0, 15
    return ((x - 8) * 0.25).to(dtype)


def _reference(q, k, v, group):
    """O, LSE in fp64 and the bounds of kv_util.attend64 for q [hq, d] over rows k, v [n, hkv, d] of 16 levels 1/4."""
    n, hkv, d = k.shape
    g = q.shape[0] // hkv
    qd, kd, vd = q.double().view(hkv, g, d), k.double(), v.double()
    x = torch.einsum("hgd,nhd->hgn", qd, kd) / math.sqrt(d)
    p = torch.softmax(x, -1)
    o = torch.einsum("hgn,nhd->hgd", p, vd)
    ds = (d + 16) * 2.0 ** -24 / math.sqrt(d) * (15 * 0.25 + 2) * qd.abs().sum(-1) + 2.0 ** -22 * x.abs().amax(-1)
    e = (2 * ds + 2.0 ** -20)[..., None]
    # |v| and the centred part scale |code - 8| coincide here (the smallest value is -8 levels)
    mag = torch.einsum("hgn,nhd->hgd", p, vd.abs())
    half = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -11
    tol = half * o.abs() + 2.0 ** -11 * mag + e * (mag + o.abs()) + 2.0 ** -19 * mag
    lse = torch.logsumexp(x, -1)
    return (o.reshape(-1, d), lse.reshape(-1), tol.reshape(-1, d),
            (e[..., 0] + 2.0 ** -21 * (1 + lse.abs())).reshape(-1))


def _check(o, lse, ref):
    ro, rl, ot, lt = ref
    assert ((o.double() - ro).abs() <= ot).all(), float((o.double() - ro).abs().max())
    assert ((lse.double() - rl).abs() <= lt).all(), float((lse.double() - rl).abs().max())


@pytest.mark.parametrize("dtype,d,group", [(torch.float16, 128, 128), (torch.bfloat16, 64, 32)])
def test_long_sequence_in_one_append(dtype, d, group):
    """150 001 keys of one KV head, cut over many CTAs; gathered back exactly."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    n, hkv, hq, ps = 150001, 1, 4, 256
    k, v = (_exact_rows(n, hkv, d, group, dtype, gen) for _ in range(2))
    pages = -(-n // ps)
    table = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)[None]
    cache = torch.zeros((pages, hkv, fa_kvcache_int4_page_bytes(ps, d, group)), dtype=torch.uint8, device=DEV)
    kw = dict(group=group, block_table=table, seqlens_k=ints([n]))
    fa_kv_append_int4(k, v, cache, **kw)
    kb, vb = fa_kv_gather_int4(cache, total=n, d=d, dtype=dtype, **kw)
    assert torch.equal(kb, k) and torch.equal(vb, v)
    q = torch.randn((1, hq, d), generator=gen, device=DEV).to(dtype)
    o, lse = fa_fwd_kvcache_int4(q, cache, **kw)
    assert fa_sync_status() == 0
    _check(o[0], lse[0], _reference(q[0], k, v, group))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,hq,hkv", [(64, 16, 16), (128, 5, 3), (128, 32, 8), (256, 0, 1), (256, 7, 2)])
def test_every_row_at_every_number_of_tokens(d, hq, hkv, interleaved):
    """From 3 tokens, each row of which gets a warp, to 23000, whose rows are all one warp's: with a rotation that leaves
    every row as it is (cosines 1, sines 0) every row gets to its place, in both caches and back."""
    gen = torch.Generator(device=DEV).manual_seed(d + hq)
    dtype, group, ps = torch.bfloat16, 64, 128
    for n in (3, 45, 310, 777, 1200, 1900, 2600, 4100, 6001, 9500, 23000):
        cut = n // 3
        lens, cu = ints([cut + 5, n - cut]), ints([0, cut, n])  # the first sequence: behind five older keys
        k, v = (_exact_rows(n, hkv, d, group, dtype, gen) for _ in range(2))
        q = _exact_rows(n, hq, d, group, dtype, gen) if hq else None
        width = -(-(n + 5) // ps)
        pages = 2 * width
        table = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).view(2, width)
        cos_sin = torch.zeros((n + 5, 32), device=DEV)
        cos_sin[:, :16] = 1
        kw = dict(block_table=table, seqlens_k=lens, cu_seqlens=cu)
        more = dict(q=q, cos_sin=cos_sin, interleaved=interleaved)
        kc, vc = (torch.zeros((pages, ps, hkv, d), dtype=dtype, device=DEV) for _ in range(2))
        got = fa_kv_append(k, v, kc, vc, **kw, **more)
        assert got is None if q is None else torch.equal(got, q)
        pos = torch.cat([torch.arange(cut, device=DEV) + 5, torch.arange(n - cut, device=DEV)])
        seq = (torch.arange(n, device=DEV) >= cut).long()
        page = table[seq, pos // ps].long()
        assert torch.equal(kc[page, pos % ps], k) and torch.equal(vc[page, pos % ps], v)
        cache = torch.zeros((pages, hkv, fa_kvcache_int4_page_bytes(ps, d, group)), dtype=torch.uint8, device=DEV)
        got = fa_kv_append_int4(k, v, cache, group=group, **kw, **more)
        assert got is None if q is None else torch.equal(got, q)
        kb, vb = fa_kv_gather_int4(cache, group=group, total=n, d=d, dtype=dtype, **kw)
        assert fa_sync_status() == 0
        assert torch.equal(kb, k) and torch.equal(vb, v), n


def test_caches_past_4_gb():
    """Pages at both ends of caches of 5 GB (4-bit) and of 2 x 5 GB (16-bit)."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    dtype, d, group, hkv, ps, n = torch.bfloat16, 128, 64, 8, 64, 150
    size = fa_kvcache_int4_page_bytes(ps, d, group)
    pages = 5 * 10 ** 9 // (size * hkv)
    cache = torch.empty((pages, hkv, size), dtype=torch.uint8, device=DEV)
    k, v = (_exact_rows(n, hkv, d, group, dtype, gen) for _ in range(2))
    table = ints([[pages - 1, 0, pages - 7]])
    kw = dict(group=group, block_table=table, seqlens_k=ints([n]))
    fa_kv_append_int4(k, v, cache, **kw)
    kb, vb = fa_kv_gather_int4(cache, total=n, d=d, dtype=dtype, **kw)
    q = torch.randn((1, 16, d), generator=gen, device=DEV).to(dtype)
    o, lse = fa_fwd_kvcache_int4(q, cache, **kw)
    assert fa_sync_status() == 0
    assert torch.equal(kb, k) and torch.equal(vb, v)
    _check(o[0], lse[0], _reference(q[0], k, v, group))
    del cache
    pages = 5 * 10 ** 9 // (ps * hkv * d * 2)
    kc, vc = (torch.empty((pages, ps, hkv, d), dtype=dtype, device=DEV) for _ in range(2))
    table = ints([[pages - 1, 0, pages - 7]])
    fa_kv_append(k, v, kc, vc, block_table=table, seqlens_k=ints([n]))
    assert fa_sync_status() == 0
    at = torch.arange(n, device=DEV)
    assert torch.equal(kc[table[0].long()[at // ps], at % ps], k)
    assert torch.equal(vc[table[0].long()[at // ps], at % ps], v)


def test_one_page_for_a_sequence_and_one_row_for_all():
    """A page of 6400 keys; a table row shared by every sequence (row stride 0), each reading a prefix."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    dtype, d, group, hkv, ps, n = torch.bfloat16, 128, 128, 2, 6400, 9000
    k, v = (_exact_rows(n, hkv, d, group, dtype, gen) for _ in range(2))
    cache = torch.zeros((3, hkv, fa_kvcache_int4_page_bytes(ps, d, group)), dtype=torch.uint8, device=DEV)
    fa_kv_append_int4(k, v, cache, group=group, block_table=ints([[2, 0]]), seqlens_k=ints([n]))
    lens = [9000, 1, 6400, 6401, 77]
    table = ints([2, 0])[None].expand(len(lens), 2)
    assert table.stride(0) == 0
    q = torch.randn((len(lens), 4, d), generator=gen, device=DEV).to(dtype)
    o, lse = fa_fwd_kvcache_int4(q, cache, group=group, block_table=table, seqlens_k=ints(lens))
    assert fa_sync_status() == 0
    for i, m in enumerate(lens):
        _check(o[i], lse[i], _reference(q[i], k[:m], v[:m], group))


def test_table_views_end_where_they_end():
    """A view of a wider table: pages past its width are not read, whatever stands there."""
    dtype, d, group, ps = torch.float16, 64, 64, 64
    cache = torch.zeros((4, 1, fa_kvcache_int4_page_bytes(ps, d, group)), dtype=torch.uint8, device=DEV)
    wide = ints([[0, 1, 2, 3], [3, 2, 1, 0]])[:, :2]
    q = torch.ones((2, 2, d), dtype=dtype, device=DEV)
    go = lambda lens: fa_fwd_kvcache_int4(q, cache, group=group, block_table=wide, seqlens_k=ints(lens))  # noqa: E731
    go([128, 128])
    assert fa_sync_status() == 0
    go([128, 129])
    assert fa_sync_status() == 6
    k = torch.ones((2, 1, d), dtype=dtype, device=DEV)
    before = cache.clone()
    fa_kv_append_int4(k, k, cache, group=group, block_table=wide, seqlens_k=ints([129, 129]))
    assert fa_sync_status() == 6 and torch.equal(cache, before)
    kc = torch.zeros((4, ps, 1, d), dtype=dtype, device=DEV)
    fa_kv_append(k, k, kc, kc.clone(), block_table=wide, seqlens_k=ints([129, 128]))
    assert fa_sync_status() == 6
    assert kc.count_nonzero() == d and bool((kc[2, 63] == 1).all())  # the second sequence's token alone


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, give what they give alone."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    dtype, d, group, hkv, ps, n = torch.bfloat16, 128, 128, 4, 64, 5000
    pages = -(-n // ps) * 2
    cache = torch.zeros((pages, hkv, fa_kvcache_int4_page_bytes(ps, d, group)), dtype=torch.uint8, device=DEV)
    k, v = (_exact_rows(2 * n, hkv, d, group, dtype, gen) for _ in range(2))
    kw = dict(group=group, block_table=torch.arange(pages, dtype=torch.int32, device=DEV).view(2, -1),
              seqlens_k=ints([n, n - 3]))
    fa_kv_append_int4(k, v, cache, **kw)
    q = torch.randn((2, 16, d), generator=gen, device=DEV).to(dtype)
    want = fa_fwd_kvcache_int4(q, cache, **kw)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for st in streams:
            got.append(fa_fwd_kvcache_int4(q, cache, stream=st, **kw))
    torch.cuda.synchronize()
    assert fa_sync_status() == 0
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
