"""pq2_attn_decode against the definition in 64 bits (bounds in attn_util)."""
import math
import threading

import pytest
import torch

from ternary_weight_int8_gb300 import pq2
import attn_util as A
import gpu_util as U

pytestmark = pytest.mark.gpu

BF16, F16, F32, I8 = A.BF16, A.F16, A.F32, A.I8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pq2.lib()
    yield
    torch.cuda.synchronize()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(q, cache, table, lens, dense, scale=None, **more):
    B, T, Hq, D = q.shape
    out, back, guard = U.guarded(q.shape, q.dtype)
    lse, lback, lguard = U.guarded(q.shape[:-1], F32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pq2.pq2_attn_decode(q, cache, table, ints(lens), scale=scale, out=out, lse=lse, status=status,
                        **more)
    torch.cuda.synchronize()
    assert not int(status)
    assert U.guards_intact(back, guard) and U.guards_intact(lback, lguard)
    verify(out, lse, q, cache, lens, dense, scale)
    again = pq2.pq2_attn_decode(q, cache, table, ints(lens), scale=scale)
    assert torch.equal(again, out)
    return out


def verify(out, lse, q, cache, lens, dense, scale=None):
    B, T, Hq, D = q.shape
    H = cache.k.shape[1]
    G = Hq // H
    eight = cache.k.dtype == I8
    scale = D ** -0.5 if scale is None else scale
    for b in range(B):
        most = (lens[b] - T + 1 + torch.arange(T, device="cuda")).repeat_interleave(G)
        for h in range(H):
            at = slice(h * G, h * G + G)
            k, v = dense[b][0][h], dense[b][1][h]
            ref = A.attend(q[b, :, at].double().reshape(T * G, D), k, v, most, scale)
            small = None
            if eight:
                n = most.clamp(0, lens[b])
                small = (2 * 0.025 * 127 * n.double())[:, None]
            A.check_rows(out[b, :, at].reshape(T * G, D),
                         None if lse is None else lse[b, :, at].reshape(T * G), ref, D,
                         F16 if eight else q.dtype, small)


def queries(B, T, Hq, D, dtype, seed):
    return torch.randn((B, T, Hq, D), generator=A.gen(seed), device="cuda").to(dtype)


KINDS = [(BF16, BF16), (F16, F16), (BF16, I8), (F16, I8)]


@pytest.mark.parametrize("dtype,cache_dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,H,G,T,page", [
    ([1], 1, 1, 1, 16), ([2], 8, 5, 1, 16), ([15, 16, 17], 2, 4, 1, 16),
    ([63, 64, 65, 0], 3, 6, 1, 32), ([127, 128, 129, 130], 1, 8, 1, 64),
    ([500, 3, 1000], 2, 16, 1, 48), ([257], 2, 17, 1, 128), ([90, 0, 1], 1, 40, 1, 16),
    ([300, 2, 5, 1], 2, 3, 4, 16), ([70, 8], 3, 1, 8, 32), ([40, 1, 7], 2, 6, 7, 16),
    ([2100], 4, 5, 2, 64), ([33], 1, 1, 64, 16)])
def test_values(dtype, cache_dtype, D, lens, H, G, T, page):
    cache, table, dense = A.make_cache(len(lens), lens, H, page, D, cache_dtype, seed=len(lens) + D)
    check(queries(len(lens), T, H * G, D, dtype, seed=G), cache, table, lens, dense)


@pytest.mark.parametrize("dtype,cache_dtype", KINDS)
@pytest.mark.parametrize("B,longest,H,G,D", [(1, 20000, 1, 1, 128), (1, 9001, 8, 5, 128),
                                             (70, 700, 4, 6, 64), (300, 90, 2, 4, 128),
                                             (5, 5000, 2, 6, 256), (400, 17, 8, 2, 64)])
def test_batches(dtype, cache_dtype, B, longest, H, G, D):
    """Ragged batches, empty sequences among them: sequences that several CTAs
    share and CTAs that several sequences share."""
    lens = [(longest * (7 * b + 3) * (7 * b + 3) // 11) % (longest + 1) for b in range(B)]
    lens[0] = longest
    cache, table, dense = A.make_cache(B, lens, H, 32, D, cache_dtype, seed=B)
    check(queries(B, 1, H * G, D, dtype, seed=B), cache, table, lens, dense)


@pytest.mark.parametrize("layout", ["heads", "tokens", "both", "gaps"])
@pytest.mark.parametrize("cache_dtype", [BF16, I8])
def test_layouts_and_strides(layout, cache_dtype):
    lens = [70, 33, 0, 200]
    cache, table, dense = A.make_cache(4, lens, 3, 32, 128, cache_dtype, seed=9, layout=layout)
    wide = torch.full((4, 2, 15 * 128 + 64), float("nan"), dtype=BF16, device="cuda")
    q = wide[..., 62:62 + 15 * 128].unflatten(-1, (15, 128))
    q.copy_(queries(4, 2, 15, 128, BF16, seed=1))
    padded = torch.full((4, table.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    padded[:, :table.shape[1]] = table
    check(q, cache, padded[:, :table.shape[1]], lens, dense)
    by_head = queries(4, 15, 2, 128, BF16, seed=2).transpose(1, 2)
    check(by_head, cache, table, lens, dense)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 4.0])
@pytest.mark.parametrize("cache_dtype", [F16, I8])
def test_scales_of_the_scores(scale, cache_dtype):
    """From the plain mean to a softmax that one key takes alone."""
    lens = [600, 45]
    cache, table, dense = A.make_cache(2, lens, 2, 16, 64, cache_dtype, seed=3)
    check(queries(2, 1, 8, 64, F16, seed=4), cache, table, lens, dense, scale=scale)


@pytest.mark.parametrize("cache_dtype", [BF16, I8])
@pytest.mark.parametrize("order", ["rising", "falling", "late", "equal"])
def test_orders_of_the_scores(cache_dtype, order):
    """Maxima that rise with every key, fall, or come last."""
    n, D = 700, 128
    cache, table, dense = A.make_cache(1, [n], 1, 16, D, BF16, seed=6)
    j = torch.arange(n, device="cuda").double()
    size = {"rising": j / n * 40, "falling": 40 - j / n * 40,
            "late": torch.where(j == n - 1, 60.0, 0.0).double(), "equal": j * 0 + 3}[order]
    k = torch.zeros((n, 1, D), device="cuda")
    k[:, 0, 0] = size.float()
    v = torch.randn((n, 1, D), generator=A.gen(8), device="cuda")
    cache = pq2.kv_cache(64, 1, 16, D, cache_dtype)
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    pq2.pq2_kv_store(k, v, cache, table, ints([n]))
    dense = [[x.double().transpose(0, 1)
              for x in pq2.pq2_kv_load(cache, table, ints([n]), tokens=n, out_dtype=F32)]]
    q = torch.zeros((1, 1, 4, D), dtype=BF16, device="cuda")
    q[..., 0] = torch.tensor([1.0, 0.5, -1.0, 0.0])
    check(q, cache, table, [n], dense, scale=1.0)


def test_an_8_bit_cache_with_scales_far_apart():
    """Values whose scales lie 2^60 apart, and none at all."""
    n, D, H = 200, 128, 2
    g = A.gen(1)
    cache = pq2.kv_cache(16, H, 16, D)
    table = torch.arange(16, dtype=torch.int32, device="cuda")[None]
    k = torch.randn((n, H, D), generator=g, device="cuda")
    v = torch.randn((n, H, D), generator=g, device="cuda")
    v[:100] *= 2.0 ** -60
    v[50] = 0
    pq2.pq2_kv_store(k, v, cache, table, ints([n]))
    k, v = (x.double().transpose(0, 1)
            for x in pq2.pq2_kv_load(cache, table, ints([n]), tokens=n, out_dtype=F32))
    q = queries(1, 1, 2 * H, D, BF16, seed=2)
    for m in (100, 101, 200):
        out = pq2.pq2_attn_decode(q, cache, table, ints([m]))
        for h in range(2 * H):
            o, _, a, *_ = A.attend(q[0, :, h].double(), k[h // 2], v[h // 2],
                                   torch.tensor([m], device="cuda"), D ** -0.5)
            # sums of terms a far larger one of which may stand alone
            assert bool(((out[0, :, h].double() - o).abs() <= 2.0 ** -7 * a + 2.0 ** -18 * a.max())
                        .all())


@pytest.mark.parametrize("cache_dtype", [BF16, I8])
def test_infinity_and_nan_where_they_are_seen(cache_dtype):
    """A key that is NaN makes the rows that see it NaN, and no others."""
    lens = [40, 40]
    cache, table, dense = A.make_cache(2, lens, 2, 16, 64, cache_dtype, seed=3)
    page, slot = int(table[0, 2]), 7  # position 39 of sequence 0
    bad = cache.k_scales if cache_dtype == I8 else cache.k
    bad[page, 1, slot] = float("nan")
    q = queries(2, 2, 4, 64, BF16, seed=1)
    out = pq2.pq2_attn_decode(q, cache, table, ints(lens))
    assert bool(out[0, 1, 2:].isnan().all())
    assert not bool(out[0, 0].isnan().any() or out[0, 1, :2].isnan().any() or out[1].isnan().any())


@pytest.mark.parametrize("dtype,cache_dtype", KINDS)
@pytest.mark.parametrize("n", [40, 3000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_of_positions_that_only_later_tokens_see(dtype, cache_dtype, n, bad):
    """The newest position's value is not finite: the tokens before it do not see
    it, whatever slice, part or join it passes through."""
    lens = [n, 29]
    cache, table, dense = A.make_cache(2, lens, 2, 16, 64, cache_dtype, seed=3)
    page, slot = int(table[0, (n - 1) // 16]), (n - 1) % 16
    if cache_dtype == I8:
        cache.v_scales[page, 1, slot] = bad
    else:
        cache.v[page, 1, slot, 5:9] = bad
    q = queries(2, 3, 8, 64, dtype, seed=1)
    out = pq2.pq2_attn_decode(q, cache, table, ints(lens))
    assert not bool(out[0, 2, 4:, 5:9].isfinite().any())
    clean = [[x.clone() for x in d] for d in dense]
    for b, rows in ((0, slice(0, 2)), (1, slice(0, 3))):
        T = rows.stop
        verify(out[b:b + 1, rows].contiguous(), None, q[b:b + 1, rows], cache,
               [lens[b] - 3 + T], [[x[:, :lens[b] - 3 + T] for x in clean[b]]])


def test_pages_outside_the_cache_read_as_zeros():
    lens = [64, 50]
    cache, table, dense = A.make_cache(2, lens, 2, 16, 64, BF16, seed=3)
    table[0, 1], table[1, 3] = -5, 1 << 20
    for b, first, last in ((0, 16, 32), (1, 48, 50)):
        for x in dense[b]:
            x[:, first:last] = 0
    check(queries(2, 1, 4, 64, BF16, seed=1), cache, table, lens, dense)


def test_lengths_behind_the_table():
    """Positions that the table does not reach read as zeros too."""
    cache, table, dense = A.make_cache(1, [48], 1, 16, 64, F16, seed=3)
    dense = [[torch.cat([x, torch.zeros((1, 30, 64), device="cuda").double()], 1)
              for x in dense[0]]]
    check(queries(1, 1, 4, 64, F16, seed=1), cache, table, [78], dense)


def test_three_dimensions_streams_and_a_captured_graph():
    lens = [300, 77, 5]
    cache, table, dense = A.make_cache(3, lens, 2, 16, 128, I8, seed=2)
    q = queries(3, 1, 8, 128, BF16, seed=1)
    want = check(q, cache, table, lens, dense)
    assert torch.equal(pq2.pq2_attn_decode(q[:, 0], cache, table, ints(lens)), want[:, 0])
    side = torch.cuda.Stream()
    n = ints(lens)
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    with torch.cuda.stream(side):
        for _ in range(5):
            outs.append(pq2.pq2_attn_decode(q, cache, table, n))
    here = [pq2.pq2_attn_decode(q, cache, table, n) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs + here)
    static_q, out = q.clone(), torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pq2.pq2_attn_decode(static_q, cache, table, n, out=out)
    for new in ([299, 1, 0], [16, 77, 2]):
        n.copy_(ints(new))
        static_q.copy_(queries(3, 1, 8, 128, BF16, seed=new[0]))
        graph.replay()
        torch.cuda.synchronize()
        short = [[x[:, :m] for x in d] for d, m in zip(dense, new)]
        verify(out, None, static_q, cache, new, short)


@pytest.mark.parametrize("B,H,G,T", [(1, 1, 1, 1), (3, 5, 4, 1), (9, 4, 3, 1), (20, 3, 6, 1),
                                     (40, 2, 5, 4), (90, 2, 16, 1), (60, 8, 2, 2)])
@pytest.mark.parametrize("cache_dtype", [BF16, I8])
def test_short_tables(B, H, G, T, cache_dtype):
    """From one item to several for every SM: clusters of 8, 4, 2 and 1, and, where
    the items would take them four rounds (480), even shares."""
    lens = [(13 * b * b + 5 * b) % 257 for b in range(B)]
    cache, table, dense = A.make_cache(B, lens, H, 16, 128, cache_dtype, seed=B, width=17)
    nbytes = pq2.lib().pq2_attn_decode_workspace_bytes(B, T, H * G, H, 128, 17 * 16)
    assert (nbytes > 0) == (B * H == 480)
    check(queries(B, T, H * G, 128, BF16, seed=G), cache, table, lens, dense)


@pytest.mark.parametrize("T,G", [(17, 1), (3, 6), (4, 6), (5, 5), (2, 23)])
@pytest.mark.parametrize("q_dtype,cache_dtype", [(BF16, BF16), (F16, F16), (F16, I8), (BF16, I8)])
def test_rows_of_256(T, G, q_dtype, cache_dtype):
    """17 to 24 rows and the first above, in clusters and in even shares."""
    lens = [0, T - 1, 100, 1333, 3000]
    cache, table, dense = A.make_cache(5, lens, 2, 16, 256, cache_dtype, seed=T)
    q = queries(5, T, 2 * G, 256, q_dtype, seed=G)
    check(q, cache, table, lens, dense)
    wide = torch.full((5, 10000), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    assert pq2.lib().pq2_attn_decode_workspace_bytes(5, T, 2 * G, 2, 256, 160000)
    check(q, cache, wide, lens, dense)


def test_graphs_replayed_at_once():
    """Two graphs of one stream, with workspaces, replayed on two streams."""
    lens = [9000, 4000, 77]
    cache, table, dense = A.make_cache(3, lens, 2, 16, 128, I8, seed=2, width=20000)
    n = ints(lens)
    qs = [queries(3, 1, 8, 128, BF16, seed=s) for s in (1, 2)]
    want = [check(q, cache, table, lens, dense) for q in qs]
    graphs, outs = [], []
    for q in qs:
        outs.append(torch.empty_like(q))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(20):
                pq2.pq2_attn_decode(q, cache, table, n, out=outs[-1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s, o in zip(graphs, streams, outs):
            with torch.cuda.stream(s):
                o.zero_()
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_two_threads_on_one_stream():
    """Each call's workspace is its own until its second kernel has run."""
    lens = [9000, 4000, 77]
    cache, table, dense = A.make_cache(3, lens, 2, 16, 128, I8, seed=2, width=20000)
    n = ints(lens)
    qs = [queries(3, 1, 8, 128, BF16, seed=s) for s in (1, 2)]
    want = [check(q, cache, table, lens, dense) for q in qs]
    torch.cuda.synchronize()
    got = [None, None]

    def calls(i):
        got[i] = [pq2.pq2_attn_decode(qs[i], cache, table, n) for _ in range(200)]

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for some, w in zip(got, want):
        assert some and all(torch.equal(o, w) for o in some)


def test_offsets_beyond_32_bits():
    """A pool whose pages lie more than 2^31 elements apart."""
    D, page, n = 64, 16, 40
    far = (1 << 31) // 2 + 64
    cache, table, dense = A.make_cache(1, [n], 1, page, D, BF16, seed=4, spare=0)
    wide = []
    for t in cache[:2]:
        back = torch.zeros((2 * far + page * D,), dtype=BF16, device="cuda")
        view = back.as_strided((3, 1, page, D), (far, page * D, D, 1))
        view.copy_(t)
        wide.append(view)
    check(queries(1, 1, 2, D, BF16, seed=3), pq2.KVCache(*wide), table, [n], dense)


def test_a_workspace_of_the_callers():
    lens = [4500, 2]
    cache, table, dense = A.make_cache(2, lens, 2, 16, 128, F16, seed=2)
    q = queries(2, 1, 10, 128, F16, seed=1)
    wide = torch.full((2, 4000), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    table = wide
    nbytes = pq2.lib().pq2_attn_decode_workspace_bytes(2, 1, 10, 2, 128, 16 * table.shape[1])
    assert nbytes
    back = torch.full((nbytes + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    check(q, cache, table, lens, dense, workspace=back[256:256 + nbytes])
    assert bool((back[:256] == 0x5A).all()) and bool((back[256 + nbytes:] == 0x5A).all())
    with pytest.raises(pq2.Pq2Error):
        pq2.pq2_attn_decode(q, cache, table, ints(lens), workspace=back[256:256 + nbytes - 16])


@pytest.mark.parametrize("dtype,cache_dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,H,G,T", [([4096], 8, 5, 1), ([4000, 0, 1, 700], 4, 3, 1),
                                        ([1, 2, 3, 2000, 513], 3, 6, 4), ([1025], 1, 8, 7)])
def test_a_wider_table_changes_nothing(dtype, cache_dtype, D, lens, H, G, T):
    """Short tables run in clusters of 1 to 8 CTAs, long ones in even shares of the
    SMs: all against 64 bits, and within two roundings of each other."""
    B = len(lens)
    cache, table, dense = A.make_cache(B, lens, H, 32, D, cache_dtype, seed=D + T, width=128)
    q = queries(B, T, H * G, D, dtype, seed=4)
    a = check(q, cache, table, lens, dense)
    for width in (300, 1000, 10000):
        wide = torch.full((B, width), -3, dtype=torch.int32, device="cuda")
        wide[:, :128] = table
        b = check(q, cache, wide, lens, dense)
        assert float((a.float() - b.float()).abs().max()) <= \
            2.0 ** -6 * float(a.float().abs().max())
