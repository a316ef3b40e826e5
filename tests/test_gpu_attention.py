"""GPU: fp8blk_paged_attn and fp8blk_latent_attn against their plain form in 64 bits."""
import numpy as np
import pytest
import torch

from attention_plain import DEV, Call, Paged, assert_attends, attend

pytestmark = pytest.mark.gpu

WIDTHS = [(64, 64), (128, 128), (192, 128), (256, 256), (512, None), (576, None)]  # None: a latent cache
IDS = ["64", "128", "192+128", "256", "latent512", "latent576"]


def _heads(v, group, kv=2):
    return (1, group) if v is None else (kv, kv * group)


def _setup(gpu, seed, lens, new, k, v, group, kv=2, page=16, e4m3=False, layout="slots", **kw):
    rng = np.random.default_rng(seed)
    kv, heads = _heads(v, group, kv)
    return Call(gpu, rng, Paged(gpu, rng, lens, kv, k, v, page, e4m3 and v is not None, layout), new, heads, **kw)


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("group", [1, 3, 8, 20])
@pytest.mark.parametrize("e4m3", [False, True])
def test_single_tokens(gpu, k, v, group, e4m3):
    """Lengths from one token, around the edges of tiles and pages, to several hundred."""
    if e4m3 and v is None:
        pytest.skip("latent caches are bf16")
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255, 257, 700]
    for page, sinks in ((1, False), (16, True), (128, False)):
        what = f"{k} {v} group {group} e4m3 {e4m3} page {page}"
        print(what, flush=True)
        c = _setup(gpu, group + page, lens, [1] * len(lens), k, v, group, page=page, e4m3=e4m3, sinks=sinks, behind=2, before=1)
        c.run()
        c.check(what)


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 37, 1000])
@pytest.mark.parametrize("new", [[2, 5, 1, 3, 4], [16, 7, 0, 1, 16], [1, 40, 17, 130, 0], [65, 333, 64, 1, 20]], ids=["few", "panel", "chunk", "long"])
def test_panels_and_chunks(gpu, k, v, causal, window, new):
    lens = [2, 77, 64, 500, 333]
    lens = [max(a, b) for a, b in zip(lens, new)]
    i = window + len(new) + new[1]
    for group, page, e4m3 in ((4, 16, False), (5, 64, True)):
        what = f"{k} {v} causal {causal} window {window} new {new} group {group} e4m3 {e4m3}"
        print(what, flush=True)
        c = _setup(gpu, i, lens, new, k, v, group, kv=1 + i % 2, page=page, e4m3=e4m3, causal=causal, window=window, sinks=bool(i % 2), behind=3)
        c.run()
        c.check(what)


@pytest.mark.parametrize("k,v,group,e4m3", [(128, 128, 8, False), (128, 128, 8, True), (64, 64, 5, False), (256, 256, 1, False), (576, None, 16, False),
                                            (576, None, 128, False), (512, None, 40, False)])
@pytest.mark.parametrize("new", [[1], [3, 1], [16]])
def test_long_caches(gpu, k, v, group, e4m3, new):
    """Enough keys to be split over workgroups, one sequence much longer than the other."""
    lens = [9001, 130][:len(new)]
    c = _setup(gpu, 3, lens, new, k, v, group, kv=1, page=64, e4m3=e4m3, sinks=True)
    c.run()
    c.check(f"{k} {v} {group} {e4m3} {new}")


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [1, 8, 16, 64])
def test_chunks_of_long_caches(gpu, k, v, e4m3, page):
    """Few tiles of rows, their keys split over workgroups; many, which are not; windows that end inside a split; small and large pages."""
    if e4m3 and v is None:
        pytest.skip("latent caches are bf16")
    for lens, new, group, window in (([5001, 700], [40, 17], 8, 0), ([3000], [300], 4, 700), ([1700, 64, 900], [200, 1, 200], 16, 0)):
        what = f"{k} {v} e4m3 {e4m3} page {page} new {new}"
        print(what, flush=True)
        c = _setup(gpu, 16, lens, new, k, v, group, kv=2, page=page, e4m3=e4m3, sinks=window > 0, window=window, behind=1)
        c.run()
        c.check(what)


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("max_new", [1, 5, 80])
def test_rows_that_see_nothing(gpu, k, v, max_new):
    """No keys at all, more new tokens than keys, pages that are none; with sinks and without."""
    for sinks in (False, True):
        lens, new = [0, 3, 0, 40], [1, max_new, 0, 1]
        c = _setup(gpu, 4, lens, new, k, v, 2, sinks=sinks, behind=1)
        c.run()
        c.check(f"{k} {max_new} {sinks}")
        assert (c.out[0] == 0).all()
        if max_new > 3:
            assert (c.out[1:1 + max_new - 3] == 0).all()


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("T", [1, 7, 50])
def test_pages_that_are_none(gpu, k, v, T):
    """A page outside of the cache, in the middle and at the end, and a sequence longer than its table."""
    for bad in (-1, 10 ** 6, -2 ** 31):
        c = _setup(gpu, 5, [150, 90], [T, T], k, v, 3, page=16)
        c.paged.table[0, [2, 5, 9]] = bad
        c.paged.table[1, :] = bad
        c.run()
        assert (c.out[T:2 * T] == 0).all()
        pages = c.paged.table[0].clone()
        c.paged.table[0, [2, 5, 9]] = 0
        kk, vv = c.paged.rows(0)
        c.paged.table[0] = pages
        absent = torch.zeros(150, dtype=torch.bool, device=DEV)
        for p in (2, 5, 9):
            absent[16 * p:16 * p + 16] = True
        want, bound = attend(kk, vv, c.q[:T], 150 - T, c.scale, absent=absent)
        assert_attends(c.out[:T], want, bound, f"{k} {T} {bad}")
    c = _setup(gpu, 6, [150], [T], k, v, 3, page=16)
    table = c.paged.table
    c.paged.table = table[:, :7].contiguous()
    c.run()
    c.paged.table = table
    kk, vv = c.paged.rows(0)
    want, bound = attend(kk, vv, c.q, 150 - T, c.scale, absent=torch.arange(150, device=DEV) >= 112)
    assert_attends(c.out, want, bound, f"{k} {T} short table")


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("T", [1, 6, 90])
@pytest.mark.parametrize("odd", [float("nan"), float("inf"), float("-inf")])
def test_what_is_not_seen_does_not_touch_a_row(gpu, k, v, T, odd):
    """Keys and values that are not finite: behind a sequence, in other tokens' future, before the window; where they are seen they count."""
    L, window = 200, 100
    for e4m3 in (False, True):
        if e4m3 and (v is None or not np.isnan(odd)):
            continue
        c = _setup(gpu, 7, [L, 64], [T, 1], k, v, 2, page=16, e4m3=e4m3, window=window)
        first = L - T
        raw = torch.uint8 if e4m3 else torch.int16
        mark = torch.tensor([odd]).to(c.paged.cache_k.dtype).view(raw).to(DEV)
        caches = [t for t in (c.paged.cache_v, c.paged.cache_k if v is None else None) if t is not None]
        spots = [first - window, first + T // 2, L - 1 if T > 1 else first - window - 1]  # before the window; in some rows' future
        for n, j in enumerate(spots):
            p, i = c.paged.table[0, j // 16].long(), j % 16
            for t in caches:
                t.view(raw)[p, i, 0, 3 + 10 * n] = mark
            if n == 0 and v is not None:
                c.paged.cache_k.view(raw)[p, i, 0, 5] = mark
        c.run()
        c.check(f"{k} {T} {odd} e4m3 {e4m3}")


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("group,e4m3", [(1, False), (8, True), (12, False)])
def test_a_panels_rows_are_those_of_single_tokens(gpu, k, v, group, e4m3):
    """Bit for bit: each row of a verify panel, and the same row as a decode step of a shorter cache."""
    for L, window in ((3000, 0), (700, 50)):
        c = _setup(gpu, 8, [L, 90], [16, 9], k, v, group, kv=1, page=32, e4m3=e4m3, sinks=True, window=window)
        c.run()
        c.check("panel")
        for i in (0, 1, 7, 14, 15):
            lens = torch.tensor([L - 15 + i, 0], dtype=torch.int32, device=DEV)
            starts = torch.tensor([0, 1, 1], dtype=torch.int32, device=DEV)
            out = torch.empty_like(c.out[:1])
            c.entry(c.paged.cache, c.q[i:i + 1], c.paged.table, lens, starts, 1, c.max_len, c.scale, out, c.workspace(), True, window, c.sinks)
            assert torch.equal(out[0], c.out[i]), (L, i)


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("layout", ["heads", "shared", "wide"])
@pytest.mark.parametrize("T", [1, 70])
def test_layouts_and_strides(gpu, k, v, layout, T):
    """Pages of heads of slots, keys beside values, rows with a gap; q and out head by head and with gaps."""
    c = _setup(gpu, 9, [333, 70], [T, T], k, v, 4, page=8, e4m3=T == 1, layout=layout)
    q = torch.zeros(c.heads, c.N, k + 8, dtype=torch.bfloat16, device=DEV)
    q[..., :k] = c.q.transpose(0, 1)
    out = torch.full((c.heads, c.N, c.v_cols + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    c.entry(*c.args(c.workspace(), q.transpose(0, 1)[..., :k], out.transpose(0, 1)[..., :c.v_cols]))
    torch.cuda.synchronize()
    c.check(f"{k} {layout} {T}", out.transpose(0, 1)[..., :c.v_cols])
    assert (out[..., c.v_cols:] == 7).all()


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("T", [1, 4, 60])
def test_extreme_scores_and_sinks(gpu, k, v, T):
    """Scores of thousands, equal scores, a scale of 0 and below, sinks that are infinite or far above all."""
    for scale in (40.0, 0.0, -3.0):
        c = _setup(gpu, 10, [300], [T], k, v, 4, scale=scale, sinks=True)
        c.sinks[0], c.sinks[1], c.sinks[2] = float("inf"), float("-inf"), 500.0
        if scale == 40.0:
            c.q[0] *= 30
        c.run()
        c.check(f"{k} {T} scale {scale}")
        assert (c.out[:, 0] == 0).all()


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
def test_scores_that_are_not_finite(gpu, k, v):
    """A row of q with NaN gives NaN, one whose scores are all -inf 0, and neither touches the others."""
    for T in (1, 8, 70):
        c = _setup(gpu, 11, [200], [T], k, v, 2)
        p, i = c.paged.where(0, 200)
        c.paged.cache_k[p, i, :, 0] = 1.0
        c.q[0, 0, 9] = float("nan")
        c.q[0, 1] = 0
        c.q[0, 1, 0] = float("-inf")
        c.run()
        assert c.out[0, 0].isnan().all() and (c.out[0, 1] == 0).all()
        want, bound = attend(*c.paged.rows(0), c.q, 200 - T, c.scale)
        assert_attends(c.out[1:], want[1:], bound[1:], f"{k} {T}")
        assert_attends(c.out[:, 2:], want[:, 2:], bound[:, 2:], f"{k} {T}")


@pytest.mark.parametrize("k,v", [(256, 256), (576, None)])
@pytest.mark.parametrize("T", [1, 100])
def test_a_cache_past_32_bit_offsets(gpu, k, v, T):
    """Pages past 2^31 values and 2^32 bytes."""
    kv, heads = _heads(v, 4)
    rng = np.random.default_rng(12)
    page = 64
    pages = (2 ** 31 + 2 ** 26) // (page * kv * k)
    p = Paged(gpu, rng, [500], kv, k, v, page)
    big = [None if t is None else torch.full((pages, *t.shape[1:]), float("nan"), dtype=t.dtype, device=DEV) for t in (p.cache_k, p.cache_v)]
    p.table[0, :8] = torch.tensor([pages - 1, 0, pages - 2, pages // 2, pages - 9, 5, pages - 100, pages - 3], dtype=torch.int32, device=DEV)
    p.cache_k, p.cache_v = big
    p.fill()
    p.cache = gpu.fp8blk_cache(*big, **({"v_cols": 512} if v is None else {}))
    c = Call(gpu, rng, p, [T], heads)
    c.run()
    c.check(f"{k} {T}")


@pytest.mark.parametrize("k,v", [(128, 128), (256, 256), (576, None)])
@pytest.mark.parametrize("T", [1, 30])
def test_many_sequences(gpu, k, v, T):
    """More sequences than compute units, most without a new token."""
    lens = [max(T, 1 + (37 * i) % 150) for i in range(600)]
    new = [T * int(i % 3 == 0) for i in range(600)]
    c = _setup(gpu, 13, lens, new, k, v, 4, behind=5)
    c.run()
    c.check("many")


@pytest.mark.parametrize("k,v", [(128, 128), (192, 128), (576, None)])
@pytest.mark.parametrize("T", [1, 6, 100])
def test_captured_replayed_and_on_other_streams(gpu, k, v, T):
    """Two graphs with workspaces of their own, replayed with other lengths, tables and inputs between eager calls; every replay equals the eager call."""
    cs = [_setup(gpu, 14 + i, [1500, 400, 90], [T, 1, T], k, v, 4, page=16) for i in range(2)]
    side = torch.cuda.Stream()
    graphs = []
    for c in cs:
        with torch.cuda.stream(side):
            c.run()
        c.check("other stream")
        graph, ws = torch.cuda.CUDAGraph(), c.workspace()
        with torch.cuda.graph(graph):
            c.entry(*c.args(ws))
        graphs.append((graph, ws))
    rng = np.random.default_rng(0)
    for step in range(4):
        for c in cs:
            lens = [int(rng.integers(T, 1501)), int(rng.integers(1, 401)), int(rng.integers(T, 91)) if T < 91 else T]
            c.paged.lens = lens
            c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
            c.q.copy_((torch.randn(c.q.shape) * 1.5).bfloat16())
            c.out.fill_(7.0)
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for c in cs:
            got = c.out.clone()
            c.out.fill_(7.0)
            c.run(stream=side)
            assert torch.equal(got.view(torch.int16), c.out.view(torch.int16)), step  # NaN where a length passes what the cache holds
            if c.paged.lens[2] <= 90:
                c.check(f"replay {step}", got)


def test_prepared_calls(gpu):
    c = _setup(gpu, 15, [100, 9], [2, 1], 128, 128, 4)
    want = c.run().clone()
    c.out.fill_(7.0)
    call = gpu.prepared("fp8blk_paged_attn", *c.args(c.workspace()))
    assert call() == gpu.OK
    torch.cuda.synchronize()
    assert torch.equal(want, c.out)
