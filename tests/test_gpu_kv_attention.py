"""gdn_kv_attention against the definition in 64 bits.

The bound: a score is off by its FP32 accumulation, at most (D + 8) 2^-23 of sum |q_i k_i| scale
(`size`), so a probability by that and the exponential's 2^-22, and by its rounding to FP16, 2^-11
of itself or, below FP16's smallest normal number (2^-14, of probabilities times 2^8), 2^-33 of the
row's largest.  What the rounding leaves is relative to sum p |v| (`spread`); the sums add
2^-20 of it.  The output is rounded once."""
import math

import pytest
import torch

import kv_reference as ref
from linear_attention_recurrence_gb300 import gdn

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def make(new, lens, H, G, D, page, dtype, gen, scales=False, garbage=True, pad=0):
    """Random codes and scales; bytes behind the sequences' ends, and pages of none, are NaN."""
    need = [-(-max(n, 0) // page) for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    shape = gdn.gdn_kv_cache(pages, G, page, D, "cpu").shape
    n = page * D // 2
    cache = torch.randint(0, 256, shape, generator=gen, dtype=torch.uint8)
    cache[..., n:] = torch.randint(0x28, 0x38, cache[..., n:].shape, generator=gen, dtype=torch.uint8)
    used = torch.zeros(pages, page, dtype=torch.bool)
    for s, m in enumerate(need):
        for i in range(m):
            table[s, i] = order.pop()
            used[table[s, i], :max(0, min(page, lens[s] - i * page))] = True
    if garbage:
        sc = cache[..., n:].unflatten(-1, (page, D // 16))
        sc.copy_(torch.where(used[:, None, None, :, None], sc, torch.tensor(0x7F, dtype=torch.uint8)))
    T = sum(new)
    q = torch.randn(T + pad, H, D, generator=gen).to(TYPES[dtype])
    hs = [0.4 + torch.rand(G, generator=gen) if scales else None for _ in range(2)]
    cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32)
    return [None if x is None else x.cuda() for x in
            (q, cache, table, torch.tensor(lens, dtype=torch.int32), cu, hs[0], hs[1])]


def compare(out, lse, q, want, T, longest):
    o, l, spread, size = (x[:T] for x in want)
    D = q.shape[-1]
    eps = torch.finfo(q.dtype).eps / 2
    delta = (D + 8) * 2 ** -23 * size + 2 ** -22
    assert torch.equal(out[:T].isnan(), o.isnan())
    worst = spread.nan_to_num(0).amax(-1, keepdim=True)
    bound = eps * o.abs() + (2 ** -11 + 2 * delta[..., None] + 2 ** -20) * spread + longest * 2 ** -33 * 8 * worst + 1e-7
    err = (out[:T].double() - o).abs()
    assert bool((err <= bound)[~o.isnan()].all()), (float(err.nan_to_num(0).max()), float((err / bound).nan_to_num(0).max()))
    if lse is not None:
        got = lse[:T].double()
        assert torch.equal(got == -math.inf, l == -math.inf)
        fine = l.isfinite()
        assert bool(((got - l).abs() <= delta + 2 ** -21 * (1 + l.abs()))[fine].all())


def check(new, lens, H, G, D, page, dtype="bf16", scales=False, causal=True, window=0, cu=True, pad=0, scale=None, seed=0,
          change=None, wide=False):
    gen = torch.Generator().manual_seed(seed)
    q, cache, table, kv, bounds, ks, vs = make(new, lens, H, G, D, page, dtype, gen, scales, pad=pad)
    if change:
        change(q, cache, table, kv)
    if wide:  # queries as columns of a wider row
        row = torch.zeros(q.shape[0], (H + 1) * D + 8, dtype=q.dtype, device="cuda")
        q_ = row[:, 8:8 + H * D].unflatten(1, (H, D))
        q_.copy_(q)
    else:
        q_ = q
    T = sum(new)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    args = dict(k_scale=ks, v_scale=vs, scale=scale, causal=causal, window=window)
    gdn.gdn_kv_attention(q_, cache, table, kv, cu_seqlens=bounds if cu else None, out=out, lse=lse, **args)
    assert gdn.gdn_device_status() == 0
    want = ref.attention(q, cache, table, kv, page, cu=bounds if cu else None, **args)
    compare(out, lse, q, want, T, max(lens))
    assert bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all())
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (8, 2), (16, 1), (10, 2), (48, 16), (24, 1)])
def test_single_tokens(dtype, D, H, G):
    check([1] * 6, [1, 2, 31, 33, 64, 700], H, G, D, 16, dtype, scales=H == 8, cu=False)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_pages(page, D):
    check([1, 1, 1, 2], [page - 1, page, page + 1, 3 * page + 5], 6, 2, D, page, "fp16", scales=True)


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 1), (True, 17), (True, 500)])
@pytest.mark.parametrize("new", [[4] * 5, [1, 0, 3, 5, 2]])
def test_a_few_tokens(window, causal, new):
    check(new, [5, 40, 333, 1000, 64], 6, 2, 128, 32, "bf16", causal=causal, window=window, pad=3, wide=True)


@pytest.mark.parametrize("D,H,G", [(128, 3, 1), (64, 8, 2), (128, 16, 2), (64, 5, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("window", [0, 100])
def test_prompts(D, H, G, dtype, window):
    check([129, 1, 40, 0, 300], [129, 70, 400, 9, 777], H, G, D, 64, dtype, scales=True, window=window, pad=2)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 257, 511, 640])
def test_prompt_lengths(n):
    check([n], [n], 3, 1, 128, 16, "bf16", seed=n)


@pytest.mark.parametrize("causal", [True, False])
def test_a_piece_behind_a_long_context(causal):
    check([70], [5000], 4, 2, 128, 64, "fp16", causal=causal)


def test_a_long_context_for_one_token():
    check([1], [40001], 6, 2, 128, 64, "bf16", cu=False)


def test_rows_that_see_nothing():
    """Lengths of 0 and below, lengths below the rows (the first rows have no place), tables of no pages."""
    def holes(q, cache, table, kv):
        table[3] = -1
        table[4] = 1 << 20
    out, lse = check([1, 3, 5, 2, 1, 130], [0, -4, 2, 50, 20, 100], 3, 1, 64, 16, "bf16", change=holes)
    assert bool((out[:4] == 0).all()) and bool((lse[:4] == -math.inf).all())


def test_missing_pages_are_not_seen():
    def holes(q, cache, table, kv):
        table[0, 1] = -1
        table[1, 0] = cache.shape[0]
        table[1, 5] = -7
    check([1, 200], [100, 200], 4, 2, 128, 16, "fp16", change=holes)
    check([1, 1], [100, 200], 4, 2, 128, 16, "fp16", change=holes)


def test_lengths_behind_the_table():
    """A length that the table's row has no places for: what is there is attended."""
    def longer(q, cache, table, kv):
        kv += 100
    check([1, 150], [64, 200], 3, 1, 64, 16, "bf16", change=longer)


def test_a_nan_in_the_values_reaches_who_sees_it():
    """A later token's NaN keeps clear of the rows before it, and beyond the window."""
    def poison(q, cache, table, kv):
        n = 16 * 32
        for at in (20, 90):
            cache[table[0, at // 16], 0, 1, n + (at % 16) * 4 + 1] = 0x7F
        cache[table[0, 3], 0, 0, n + 4 * 2] = 0xFF  # a key's
    out, _ = check([120], [120], 3, 1, 64, 16, "fp16", change=poison)
    assert not bool(out[:20].isnan().any()) and bool(out[20:].isnan().all())
    out, _ = check([4], [120], 3, 1, 64, 16, "fp16", change=poison, window=27)  # places 90 .., 91 .., 92 ..
    assert bool(out[0].isnan().all()) and not bool(out[1:].isnan().any())


def test_queries_of_any_size():
    """Rows from 2^-30 to 2^30, rows of zeros; one NaN row and its neighbours."""
    def sizes(q, cache, table, kv):
        q[0] *= 2.0 ** -30
        q[1] = 0
        q[2] *= 2.0 ** 30
        q[3, 0, 0] = math.nan
    gen = torch.Generator().manual_seed(1)
    for new in ([1] * 5, [5]):
        out, _ = check(new, [60] * len(new), 3, 1, 128, 32, "bf16", change=sizes, scale=2.0 ** -20)
        assert bool(out[3, 0].isnan().all()) and not bool(out[4].isnan().any())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new", [[1] * 5, [5], [120, 5]])
def test_infinite_queries(new, dtype):
    """A row with an infinity is NaN where a score is infinite or NaN; its neighbours are as ever."""
    def infinite(q, cache, table, kv):
        q[1, 1, 7] = math.inf
        q[3, 0, 100] = -math.inf
    out, _ = check(new, [200] * len(new), 3, 1, 128, 32, dtype, change=infinite)
    assert not bool(out[[0, 2, 4]].isnan().any())
    assert bool(out[1, 1].isnan().all()) and bool(out[3, 0].isnan().all())


def test_windows_of_any_size():
    """A window beyond 32 bits is one that leaves nothing out."""
    gen = torch.Generator().manual_seed(4)
    for new, lens in (([1, 2], [40, 300]), ([150], [200])):
        q, cache, table, kv, cu, _, _ = make(new, lens, 3, 1, 64, 16, "bf16", gen)
        want = gdn.gdn_kv_attention(q, cache, table, kv, cu_seqlens=cu)
        for window in (2 ** 31 - 1, 2 ** 32 + 5, 2 ** 63 - 1):
            assert torch.equal(want, gdn.gdn_kv_attention(q, cache, table, kv, cu_seqlens=cu, window=window))
        with pytest.raises(gdn.GDNError):
            gdn.gdn_kv_attention(q, cache, table, kv, cu_seqlens=cu, window=-1)


def test_scores_of_any_size():
    check([1, 2], [300, 50], 6, 2, 128, 64, "bf16", scale=20.0)
    check([140], [300], 6, 2, 128, 64, "bf16", scale=20.0)
    check([1, 2], [300, 50], 6, 2, 128, 64, "fp16", scale=0.0)
    check([140], [300], 3, 1, 64, 64, "fp16", scale=-0.3)


def test_rows_off_boundaries():
    gen = torch.Generator().manual_seed(2)
    for new, lens in (([1, 1, 1], [40, 3, 90]), ([150], [200])):
        q, cache, table, kv, cu, _, _ = make(new, lens, 3, 1, 64, 16, "bf16", gen)
        T = sum(new)
        base = torch.zeros(T, 3 * 64 + 1, dtype=q.dtype, device="cuda")
        base[:, 1:] = q.flatten(1)
        odd = torch.zeros(T, 3 * 64 + 3, dtype=q.dtype, device="cuda")
        out = odd[:, 1:1 + 192].unflatten(1, (3, 64))
        gdn.gdn_kv_attention(base[:, 1:].unflatten(1, (3, 64)), cache, table, kv, cu_seqlens=cu, out=out)
        assert torch.equal(out, gdn.gdn_kv_attention(q, cache, table, kv, cu_seqlens=cu))
        assert not bool(odd[:, 0].any()) and not bool(odd[:, 193:].any())


def test_empty_calls():
    gen = torch.Generator().manual_seed(2)
    q, cache, table, kv, cu, _, _ = make([2], [9], 2, 1, 64, 16, "bf16", gen)
    assert gdn.gdn_kv_attention(q[:0], cache, table, kv).shape == (0, 2, 64)
    out = torch.full_like(q, 3)
    gdn.gdn_kv_attention(q, cache, table[:, :0], kv, out=out)  # no pages: nothing is seen
    assert not bool(out.any())
    out.fill_(3)
    gdn.gdn_kv_attention(q, cache, table, kv, cu_seqlens=torch.tensor([1, 5], dtype=torch.int32, device="cuda"), out=out)
    assert bool((out == 3).all())  # a bound past the rows: no sequence


def test_many_requests_and_runs_agree():
    gen = torch.Generator().manual_seed(7)
    lens = torch.randint(1, 300, (700,), generator=gen).tolist()
    first, _ = check([1] * 700, lens, 4, 2, 64, 16, "bf16", cu=False, seed=7)
    again, _ = check([1] * 700, lens, 4, 2, 64, 16, "bf16", cu=False, seed=7)
    assert torch.equal(first, again)


def test_prompts_and_single_tokens_in_one_call():
    check([1, 200, 1, 1, 30, 1], [500, 200, 3, 64, 900, 17], 6, 2, 128, 16, "bf16")


@pytest.mark.parametrize("bounds", [[0, 1], [7, 8], [3, 99], [0, 0], [0, 100], [2, 3, 40, 41]])
def test_rows_of_no_sequence_around_the_sequences(bounds):
    """A batch padded before and behind: what a sequence is goes by its bounds alone."""
    gen = torch.Generator().manual_seed(4)
    n = len(bounds) - 1
    new = [b - a for a, b in zip(bounds, bounds[1:])]
    lens = [m + 60 for m in new]
    q, cache, table, kv, _, _, _ = make(new, lens, 3, 1, 128, 16, "bf16", gen, pad=100 - sum(new))
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    gdn.gdn_kv_attention(q, cache, table, kv, cu_seqlens=cu, out=out, lse=lse)
    want = ref.attention(q, cache, table, kv, 16, cu=cu)
    inside = slice(bounds[0], bounds[-1])
    compare(out[inside], lse[inside], q, [w[inside] for w in want], sum(new), max(lens))
    outside = [*range(bounds[0]), *range(bounds[-1], 100)]
    assert bool((out[outside] == 7).all()) and bool((lse[outside] == 7).all())


@pytest.mark.parametrize("D,H,G", [(128, 3, 1), (64, 16, 2)])
def test_prompts_run_alike_whatever_the_workspace_held(D, H, G):
    """The same call twice, its workspace full of NaN in between: the same bits; on two streams at once too."""
    gen = torch.Generator().manual_seed(5)
    q, cache, table, kv, cu, ks, vs = make([200, 1, 90, 4], [4200, 900, 90, 33], H, G, D, 32, "bf16", gen, True)
    args = dict(cu_seqlens=cu, k_scale=ks, v_scale=vs)
    first = gdn.gdn_kv_attention(q, cache, table, kv, **args)
    torch.full((64 << 20,), math.nan, device="cuda")  # (freed at once: what the next call is given)
    again = gdn.gdn_kv_attention(q, cache, table, kv, **args)
    assert torch.equal(first, again)
    torch.cuda.synchronize()
    outs, streams = [], [torch.cuda.Stream() for _ in range(3)]
    for i in range(12):
        with torch.cuda.stream(streams[i % 3]):
            outs.append(gdn.gdn_kv_attention(q, cache, table, kv, **args))
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    assert gdn.gdn_device_status() == 0


def test_a_prompt_captured_and_replayed():
    gen = torch.Generator().manual_seed(6)
    q, cache, table, kv, cu, _, _ = make([150, 20], [1150, 70], 6, 2, 128, 64, "fp16", gen)
    out = torch.empty_like(q)
    want = gdn.gdn_kv_attention(q, cache, table, kv, cu_seqlens=cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_kv_attention(q, cache, table, kv, cu_seqlens=cu, out=out)
    for _ in range(3):
        out.fill_(9)
        graph.replay()
        assert torch.equal(out, want)
    q.mul_(0.5)
    graph.replay()
    assert torch.equal(out, gdn.gdn_kv_attention(q, cache, table, kv, cu_seqlens=cu))


def test_more_sequences_than_a_warp_has_lanes():
    gen = torch.Generator().manual_seed(8)
    new = torch.randint(0, 40, (70,), generator=gen).tolist()
    check(new, [n + 10 * (i % 5) + 1 for i, n in enumerate(new)], 3, 1, 128, 16, "bf16", window=33)


def test_far_pages():
    """Offsets past 32 bits."""
    dev, page, G, D = "cuda", 256, 4, 128
    n = (5 << 30) // (G * 2 * page * 9 * D // 16)
    cache = torch.empty((n, G, 2, page * 9 * D // 16), dtype=torch.uint8, device=dev)
    for T in (1, 90):
        gen = torch.Generator().manual_seed(3)
        q, small, table, kv, _, _, _ = make([T], [500], 8, G, D, page, "bf16", gen)
        cache[n - small.shape[0]:] = small
        far = torch.where(table >= 0, table + (n - small.shape[0]), table)
        assert torch.equal(gdn.gdn_kv_attention(q, cache, far, kv), gdn.gdn_kv_attention(q, small, table, kv))


def run_layer(state, x, stream=None):
    """Append, then attend: a decode or prompt step of one layer."""
    q, k, v = x
    q = gdn.gdn_kv_append(k, v, state["cache"], state["table"], state["lens"], q=q, inv_freq=state["freq"], stream=stream)
    return gdn.gdn_kv_attention(q, state["cache"], state["table"], state["lens"], stream=stream)


def layer(n, H, G, D, page, pages, dev="cuda"):
    return {"cache": gdn.gdn_kv_cache(n * pages, G, page, D, dev), "lens": torch.zeros(n, dtype=torch.int32, device=dev),
            "table": torch.randperm(n * pages, device=dev).int().view(n, pages),
            "freq": 1e4 ** (-torch.arange(0, D, 2, device=dev).float() / D)}


@pytest.mark.parametrize("D,H,G", [(128, 6, 2), (64, 8, 2)])
def test_a_prompt_and_its_tokens_one_by_one(D, H, G):
    """The run of both operators: a prompt at once, in pieces, and token by token sees the same
    cache, and gives the same rows (within both runs' bounds)."""
    gen = torch.Generator().manual_seed(1)
    n, T = 2, 150
    x = [torch.randn(n, T, h, D, generator=gen).bfloat16().cuda() for h in (H, G, G)]
    cut = lambda a, b: [y[:, a:b].reshape(-1, *y.shape[2:]) for y in x]
    results = []
    torch.manual_seed(0)
    first = layer(n, H, G, D, 16, 12)
    for pieces in ([T], [100, 50], [149, 1], [1] * T):
        st = dict(first, cache=torch.zeros_like(first["cache"]), lens=torch.zeros_like(first["lens"]))
        outs, at = [], 0
        for m in pieces:
            st["lens"] += m
            outs.append(run_layer(st, cut(at, at + m)).view(n, m, H, D))
            at += m
        results.append((torch.cat(outs, 1), st["cache"]))
    q = ref.rotate(cut(0, T)[0], torch.arange(T).repeat(n).cuda(), first["freq"], False).bfloat16()
    lens = torch.full((n,), T, dtype=torch.int32, device="cuda")
    want = ref.attention(q, results[0][1], first["table"], lens, 16)
    for out, cache in results:
        assert torch.equal(cache, results[0][1])
        # (a query's rounding to BF16 may go the other way at a tie: two half steps of its scores)
        o, _, spread, size = want
        err = (out.reshape(-1, H, D).double() - o).abs()
        bound = 2 ** -8 * o.abs() + (2 ** -11 + 2 * 2 ** -8 * 2 ** -8 * size[..., None] + 2 * 136 * 2 ** -23 * size[..., None] + 2 ** -19) * spread + 1e-6
        assert bool((err <= bound).all()), float((err / bound).max())


def test_streams_graphs_and_two_at_once():
    gen = torch.Generator().manual_seed(1)
    n, H, G, D = 9, 6, 2, 128
    torch.manual_seed(0)
    st = layer(n, H, G, D, 16, 20)
    x = [torch.randn(n, h, D, generator=gen).bfloat16().cuda() for h in (H, G, G)]
    st["lens"] += torch.randint(1, 300, (n,), generator=gen).int().cuda()
    want = run_layer(st, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run_layer(st, x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    # captured: lengths change between replays, two graphs share their memory pool
    lens = st["lens"].clone()
    pool = torch.cuda.graph_pool_handle()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            out = run_layer(st, x)
        graphs.append((graph, out))
    cache = st["cache"].clone()
    for graph, out in graphs + graphs:
        st["lens"].copy_(lens)
        st["cache"].copy_(cache)  # (the shorter lengths put the token at another place)
        graph.replay()
        assert torch.equal(out, want)
        st["lens"].copy_(lens // 2 + 1)
        graph.replay()
        short = run_layer(st, x)
        graph.replay()
        assert torch.equal(out, short)
    # two calls at once on streams of their own
    st["lens"].copy_(lens)
    st["cache"].copy_(cache)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(gdn.gdn_kv_attention(x[0], st["cache"], st["table"], st["lens"]))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, outs[0])
