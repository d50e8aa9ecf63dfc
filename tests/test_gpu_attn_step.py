"""The cache and the attention together, as a server runs a model's layer: the
qkv projection's output stored, a prompt in chunks over its prefix read back,
then decode steps over the pages, two requests sharing their first pages; all
captured as graphs as well.  Against 64 bits over what the cache stands for."""
import pytest
import torch

from ternary_weight_int8_gb300 import pq2, synth
import attn_util as A

pytestmark = pytest.mark.gpu

BF16, F32, I8 = A.BF16, A.F32, A.I8
HQ, H, D, HIDDEN, PAGE = 10, 2, 128, 1280, 16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pq2.lib()
    yield
    torch.cuda.synchronize()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def dense(cache, table, b, n):
    """What sequence b's pages stand for, [H][n][D] in 64 bits."""
    k, v = pq2.pq2_kv_load(cache, table[b:b + 1], ints([n]), tokens=n, out_dtype=F32)
    return k.double().transpose(0, 1), v.double().transpose(0, 1)


def check(out, q, k, v, most, weights):
    """out, q [rows][HQ][D] of one sequence against its keys."""
    for h in range(HQ):
        ref = A.attend(q[:, h].double(), k[h * H // HQ], v[h * H // HQ], most, D ** -0.5)
        small = (2 * 0.2 * 127 * ref[6].double())[:, None]
        A.check_rows(out[:, h], None, ref, D, weights, small)


@pytest.mark.parametrize("cache_dtype", [I8, BF16])
def test_a_layer_of_chunks_and_steps(cache_dtype):
    raw = synth.raw_weights((HQ + 2 * H) * D, HIDDEN, seed=1, device="cuda")
    codes, scales = pq2.pq2_prepare(raw, HIDDEN)
    cache = pq2.kv_cache(40, H, PAGE, D, cache_dtype)
    # Requests 0 and 1 share their first two pages; request 2 has its own.
    table = torch.full((3, 12), -1, dtype=torch.int32, device="cuda")
    table[0, :8] = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7])
    table[1, :8] = torch.tensor([0, 1, 8, 9, 10, 11, 12, 13])
    table[2, :8] = torch.tensor([20, 19, 18, 17, 16, 15, 14, 30])
    have = [0, 0, 0]

    def project(tokens, seed):
        x = synth.activations(tokens, HIDDEN, seed=seed, device="cuda", outlier_frac=0.01)
        qkv = pq2.pq2_linear(x, codes, scales, out_dtype=BF16)
        qkv = qkv / qkv.float().square().mean(1, keepdim=True).sqrt().bfloat16()
        cuts = [0, HQ * D, (HQ + H) * D, (HQ + 2 * H) * D]
        return [qkv[:, a:b].unflatten(1, (-1, D)) for a, b in zip(cuts, cuts[1:])]

    def sums(n):
        return ints([0, n[0], n[0] + n[1], n[0] + n[1] + n[2]])

    for step, new in enumerate([[32, 0, 40], [19, 25, 1], [0, 30, 33]]):
        q, k, v = project(sum(new), 10 + step)
        if step == 0:
            have[1] = 32  # the pages that request 0 writes now
        have = [a + b for a, b in zip(have, new)]
        lens = ints(have)
        pq2.pq2_kv_store(k, v, cache, table, lens, cu=sums(new))
        whole = pq2.pq2_kv_load(cache, table, lens, cu=sums(have), tokens=sum(have))
        out = pq2.pq2_attn_prefill(q, *whole, sums(new), sums(have))
        at, key = 0, 0
        for b in range(3):
            rows, n = new[b], have[b]
            if rows:
                kk, vv = (x[key:key + n].double().transpose(0, 1) for x in whole)
                most = n - rows + 1 + torch.arange(rows, device="cuda")
                check(out[at:at + rows], q[at:at + rows], kk, vv, most, BF16)
            at, key = at + rows, key + n
    # Decode steps of one and of two tokens, the same calls captured and replayed.
    lens, q_in, k_in, v_in, out = ints(have), *(torch.empty((6, n, D), dtype=BF16, device="cuda")
                                               for n in (HQ, H, H)), None
    for T in (1, 2):
        qs, ks, vs = q_in[:3 * T], k_in[:3 * T], v_in[:3 * T]

        def step():
            pq2.pq2_kv_store(ks, vs, cache, table, lens)
            return pq2.pq2_attn_decode(qs.view(3, T, HQ, D), cache, table, lens)
        for seed in (30, 31, 32):
            for x, y in zip((qs, ks, vs), project(3 * T, 10 * T + seed)):
                x.copy_(y)
            have = [n + T for n in have]
            lens.copy_(ints(have))
            if seed == 30:
                out = step()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    captured = step()
            else:
                graph.replay()
                out = captured
            torch.cuda.synchronize()
            for b in range(3):
                kk, vv = dense(cache, table, b, have[b])
                most = have[b] - T + 1 + torch.arange(T, device="cuda")
                check(out[b], qs.view(3, T, HQ, D)[b], kk, vv, most,
                      A.F16 if cache_dtype == I8 else BF16)


def test_calls_on_two_streams_at_once():
    """Two batches over one cache, each with its own stream and workspace."""
    lens = [5000, 77, 300, 4100]
    cache, table, _ = A.make_cache(4, lens, H, PAGE, D, BF16, seed=2)
    q = torch.randn((4, HQ, D), generator=A.gen(1), device="cuda").bfloat16()
    n = ints(lens)
    want = pq2.pq2_attn_decode(q, cache, table, n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(10):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(pq2.pq2_attn_decode(q, cache, table, n))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
