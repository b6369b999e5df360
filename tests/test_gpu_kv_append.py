"""gdn_kv_append against the definition in 64 bits.  Codes, scales and what k_out and v_out
receive have one right answer; rotated queries are off by the rotation's FP32 arithmetic (bound
2^-21 of a pair's size: the angle to 2^-23.3, sine and cosine to 2 ulp, three roundings) and one
rounding to their type."""
import pytest
import torch

import kv_reference as ref
from linear_attention_recurrence_gb300 import gdn

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def layout(lens, page, gen, spare=3):
    """A table of pages in no order, and how many pages there are."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    for s, n in enumerate(need):
        for i in range(n):
            table[s, i] = order.pop()
    return table, pages


def held(x, scale, dtype):
    """What the cache holds of rows x [T][G][D] (FP64): codes, scale bytes, values rounded to dtype."""
    T, G, D = x.shape
    codes = torch.zeros((T, G, D), dtype=torch.int32)
    scales = torch.zeros((T, G, D // 16), dtype=torch.int32)
    values = torch.zeros((T, G, D), dtype=torch.float64)
    for t in range(T):
        for g in range(G):
            hs = 1.0 if scale is None else float(scale[g])
            for b in range(D // 16):
                c, byte = ref.quantise(x[t, g, 16 * b:16 * b + 16].tolist(), hs)
                codes[t, g, 16 * b:16 * b + 16] = torch.tensor(c)
                scales[t, g, b] = byte
                s = float("nan") if byte == 0x7F else ref._E4M3[byte] * hs
                values[t, g, 16 * b:16 * b + 16] = torch.tensor([(-1 if v & 8 else 1) * ref.E2M1[v & 7] * s for v in c])
    return codes, scales, values


def check(dtype, new, lens, H, G, D, page, rotary, interleaved, scales, positions=None, pad=0, wide=False, cu=True,
          change=None, seed=0):
    ty = TYPES[dtype]
    gen = torch.Generator().manual_seed(seed)
    T = sum(new)
    table, pages = layout(lens, page, gen)
    q, k, v = (torch.randn(T + pad, n, D, generator=gen).to(ty) for n in (H, G, G))
    if change:
        change(k, v)
    freq = 1e4 ** (-torch.arange(0, rotary, 2).float() / max(rotary, 1))
    hs = [0.3 + torch.rand(G, generator=gen) if scales else None for _ in range(2)]
    bounds = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32)
    dev = "cuda"
    cache = torch.randint(0, 256, gdn.gdn_kv_cache(pages, G, page, D, "cpu").shape, generator=gen, dtype=torch.uint8)
    before = cache.clone()
    cache = cache.to(dev)
    if wide:  # columns of one wider row
        row = torch.cat([x.flatten(1) for x in (q, k, v)] + [torch.zeros(T + pad, 5 * 16, dtype=ty)], 1).to(dev)
        q_, k_, v_ = (row[:, a:a + n * D].unflatten(1, (n, D)) for a, n in ((0, H), (H * D, G), ((H + G) * D, G)))
    else:
        q_, k_, v_ = (x.to(dev) for x in (q, k, v))
    outs = [torch.full((T + pad, n, D), 7.0, dtype=ty, device=dev) for n in (H, G, G)]
    gdn.gdn_kv_append(k_, v_, cache, table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), q=q_,
                      inv_freq=freq.to(dev) if rotary else None, interleaved=interleaved,
                      positions=None if positions is None else positions.to(dev),
                      k_scale=None if not scales else hs[0].to(dev), v_scale=None if not scales else hs[1].to(dev),
                      cu_seqlens=bounds.to(dev) if cu else None, q_out=outs[0], k_out=outs[1], v_out=outs[2])
    torch.cuda.synchronize()
    places = torch.cat([torch.arange(n - m, n) for m, n in zip(new, lens)]) if T else torch.zeros(0, dtype=torch.long)
    pos = places if positions is None else positions[:T].long()
    eps = torch.finfo(ty).eps / 2
    # queries
    want = ref.rotate(q[:T], pos, freq, interleaved)
    half = rotary // 2
    size = torch.zeros_like(want)
    a = q[:T].double().abs()
    if interleaved:
        size[..., :rotary] = (a[..., 0:rotary:2] + a[..., 1:rotary:2]).repeat_interleave(2, -1)
    else:
        size[..., :rotary] = (a[..., :half] + a[..., half:rotary]).repeat(1, 1, 2)
    got = outs[0].double().cpu()
    err = (got[:T] - want).abs()
    assert bool((err <= eps * want.abs() + 2 ** -21 * size * (1 + eps)).all()), float(err.max())
    # keys and values, in the cache and returned
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    after = cache.cpu()
    n = page * D // 2
    touched = torch.zeros_like(after, dtype=torch.bool)
    for which, x in ((0, ref.rotate(k[:T], pos, freq, interleaved)), (1, v[:T].double())):
        codes, bytes_, values = held(x, hs[which], ty)
        assert torch.equal(outs[1 + which][:T].cpu().isnan(), values.isnan())
        # (the product of code, scale and the head's scale takes two FP32 roundings)
        assert bool(((outs[1 + which][:T].double().cpu() - values).nan_to_num(0).abs()
                     <= (eps + 2 ** -23) * values.nan_to_num(0).abs()).all())
        if not scales:
            assert torch.equal(outs[1 + which][:T].double().cpu().nan_to_num(99), values.to(ty).double().nan_to_num(99))
        for t in range(T):
            at = int(places[t])
            p = ref.page_of(table, int(seq[t]), at, page, pages)
            if p is None:
                continue
            r = at % page
            c = after[p, :, which, :n].unflatten(-1, (page, D // 2))[:, r].int()
            c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
            assert torch.equal(c, codes[t]), (t, which)
            assert torch.equal(after[p, :, which, n:].unflatten(-1, (page, D // 16))[:, r].int(), bytes_[t]), (t, which)
            touched[p, :, which, :n].unflatten(-1, (page, D // 2))[:, r] = True
            touched[p, :, which, n:].unflatten(-1, (page, D // 16))[:, r] = True
    assert torch.equal(after[~touched], before[~touched])  # nothing else
    for o in outs:  # rows of no sequence
        assert bool((o[T:] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rotary,interleaved", [(0, False), (32, False), (64, True), (128, False), (128, True)])
def test_types_and_rotations(dtype, rotary, interleaved):
    check(dtype, [3, 1, 9], [5, 40, 9], 6, 2, 128, 16, rotary, interleaved, False)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages_narrow_heads_and_scales(dtype, page):
    check(dtype, [2, 17], [page + 1, 2 * page], 3, 1, 64, page, 64, page == 32, True, pad=2)


@pytest.mark.parametrize("cu", [True, False])
@pytest.mark.parametrize("wide", [True, False])
def test_one_token_each(cu, wide):
    check("bf16", [1] * 7, [1, 2, 16, 17, 33, 100, 31], 12, 4, 128, 16, 128, False, False, cu=cu, wide=wide)


def test_odd_strides():
    """Rows that start off 16-byte boundaries."""
    dev, gen = "cuda", torch.Generator().manual_seed(3)
    G, D, T = 2, 64, 5
    base = torch.randn(T, 2 * G * D + 3, generator=gen).bfloat16().to(dev)
    k, v = base[:, 1:1 + G * D].unflatten(1, (G, D)), base[:, 2 + G * D:2 + 2 * G * D].unflatten(1, (G, D))
    args = (torch.arange(1, device=dev, dtype=torch.int32)[None], torch.tensor([T], device=dev, dtype=torch.int32))
    one, two = (gdn.gdn_kv_cache(1, G, 16, D) for _ in range(2))
    freq = torch.rand(D // 2, generator=gen).to(dev)
    qa = gdn.gdn_kv_append(k, v, one, *args, q=k, inv_freq=freq)
    qb = gdn.gdn_kv_append(k.contiguous(), v.contiguous(), two, *args, q=k.contiguous(), inv_freq=freq)
    assert torch.equal(one, two) and torch.equal(qa, qb)


def test_queries_in_place_and_none():
    dev, gen = "cuda", torch.Generator().manual_seed(4)
    G, H, D, T = 2, 4, 128, 33
    k, v = (torch.randn(T, G, D, generator=gen).half().to(dev) for _ in range(2))
    q = torch.randn(T, H, D, generator=gen).half().to(dev)
    table, lens = torch.arange(3, device=dev, dtype=torch.int32)[None], torch.tensor([T], device=dev, dtype=torch.int32)
    freq = torch.rand(D // 2, generator=gen).to(dev)
    caches = [gdn.gdn_kv_cache(3, G, 16, D) for _ in range(3)]
    want = gdn.gdn_kv_append(k, v, caches[0], table, lens, q=q, inv_freq=freq)
    got = q.clone()
    gdn.gdn_kv_append(k, v, caches[1], table, lens, q=got, inv_freq=freq, q_out=got)
    assert gdn.gdn_kv_append(k, v, caches[2], table, lens, inv_freq=freq) is None
    assert torch.equal(got, want) and torch.equal(caches[0], caches[1]) and torch.equal(caches[0], caches[2])


def test_positions_far_and_negative():
    pos = torch.tensor([0, 1, -1, 1 << 20, (1 << 31) - 1, -(1 << 31), 12345678, 7], dtype=torch.int32)
    check("fp32", [8], [8], 2, 1, 64, 16, 64, False, False, positions=pos)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_ties_zeros_infinities_and_nans(dtype):
    """Values on the borders between codes and between scales, groups of zeros, tiny groups
    (scale 0), huge ones (the largest scale), infinities, NaN."""
    def change(k, v):
        for x in (k, v):
            x[0, 0, :16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0])
            x[0, 0, 16:32] = 0
            x[0, 0, 32:48] = 6 * 1.0625 * torch.linspace(-1, 1, 16)  # between two scales
            x[0, 0, 48:64] = 0.004 * torch.linspace(-1, 1, 16)
            x[1, 0, :16] = 60000.0
            x[1, 0, 16] = float("inf")
            x[1, 0, 32] = float("nan")
            x[1, 0, 48] = -float("inf")
            x[2, 0, :] = torch.randn(64).mul(8).round() / 8  # many ties
    for scales in (False, True):
        check(dtype, [4], [4], 1, 1, 64, 16, 0, False, scales, change=change)


def test_ties_under_a_scale_of_a_power_of_two():
    gen = torch.Generator().manual_seed(9)
    v = (torch.randn(40, 1, 64, generator=gen) * 8).round().div(8).bfloat16()
    for s in (0.5, 0.75, 1.125, 0.3):
        hs = torch.tensor([s])
        cache, dev = gdn.gdn_kv_cache(3, 1, 16, 64), "cuda"
        out = torch.empty_like(v, device=dev)
        gdn.gdn_kv_append(v.to(dev), v.to(dev), cache, torch.arange(3, device=dev, dtype=torch.int32)[None],
                          torch.tensor([40], device=dev, dtype=torch.int32), v_scale=hs.to(dev), v_out=out)
        codes, _, _ = held(v.double(), hs, torch.bfloat16)
        n = 16 * 32
        c = cache[:, 0, 1, :n].unflatten(-1, (16, 32)).flatten(0, 1)[:40].int().cpu()
        assert torch.equal(torch.stack([c & 15, c >> 4], -1).flatten(-2), codes[:, 0])


def test_places_that_do_not_exist():
    """Pages below 0 or past the pool, places behind the table's row and below 0."""
    dev, gen = "cuda", torch.Generator().manual_seed(5)
    k = torch.randn(60, 1, 64, generator=gen).half().to(dev)
    table = torch.tensor([[0, -1], [7, 1], [2, 99]], device=dev, dtype=torch.int32)
    lens = torch.tensor([30, 45, 5], device=dev, dtype=torch.int32)  # 45: behind 32; 5 of 20: below 0
    cache = torch.full_like(gdn.gdn_kv_cache(3, 1, 16, 64), 0x5A)
    full = cache.clone()
    out = torch.empty_like(k)
    gdn.gdn_kv_append(k, k, cache, table, lens, q=k, q_out=out, k_out=torch.empty_like(k))
    torch.cuda.synchronize()
    changed = (cache != full).flatten(1).any(1).tolist()
    assert changed == [True, True, True]
    n = 16 * 32
    rows = [(cache[p, 0, 0, :n] != 0x5A).view(16, 32).any(1).tolist() for p in range(3)]
    assert rows[0] == [False] * 10 + [True] * 6  # places 10 .. 15 of sequence 0
    assert rows[1] == [False] * 9 + [True] * 7  # places 25 .. 31 of sequence 1 (page 7 is none)
    assert rows[2] == [True] * 5 + [False] * 11  # places 0 .. 4 of sequence 2
    assert torch.equal(out, k)


def test_no_rows_and_unsound_bounds():
    dev = "cuda"
    k = torch.ones(4, 1, 64, device=dev).half()
    table, cache = torch.zeros(2, 1, device=dev, dtype=torch.int32), gdn.gdn_kv_cache(1, 1, 16, 64)
    lens = torch.tensor([3, 3], device=dev, dtype=torch.int32)
    gdn.gdn_kv_append(k[:0], k[:0], cache, table, lens)
    gdn.gdn_kv_append(k, k, cache, table, lens, cu_seqlens=torch.tensor([-3, 2, 9], device=dev, dtype=torch.int32))
    torch.cuda.synchronize()
    assert not bool(cache.any())


def test_many_sequences():
    """More sequences than one step of the search covers, most of them empty."""
    gen = torch.Generator().manual_seed(6)
    new = [0] * 2500
    for i in (0, 3, 31, 32, 33, 1023, 1024, 2047, 2499):
        new[i] = int(torch.randint(1, 4, (1,), generator=gen))
    check("bf16", new, [n + i % 3 for i, n in enumerate(new)], 1, 1, 64, 16, 32, False, False, pad=3)


def test_far_pages():
    """Offsets past 32 bits: the last pages of a cache of 5 GB."""
    dev, page, G, D = "cuda", 256, 4, 128
    n = (5 << 30) // (G * 2 * page * 9 * D // 16)
    cache = torch.empty((n, G, 2, page * 9 * D // 16), dtype=torch.uint8, device=dev)
    cache[-2:] = 0
    small = torch.zeros_like(cache[-2:])
    k, v = (torch.randn(300, G, D, device=dev).bfloat16() for _ in range(2))
    lens = torch.tensor([300], device=dev, dtype=torch.int32)
    gdn.gdn_kv_append(k, v, cache, torch.tensor([[n - 1, n - 2]], device=dev, dtype=torch.int32), lens)
    gdn.gdn_kv_append(k, v, small, torch.tensor([[1, 0]], device=dev, dtype=torch.int32), lens)
    assert torch.equal(cache[-2:], small)
