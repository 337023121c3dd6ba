"""A paged cache: the write of new keys and values, exact, and attention over it against
the same fp64 definition, and within the same tolerances, as attention over packed keys."""
import numpy as np
import pytest
import torch

import oracle as O
from layer_wise_obs_amd import _lib as L
from tests.test_gpu_attention import _check, _i32, _randn, _starts

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


class Cache:
    """Pages of a sequence anywhere in the pool; `fill` in all that no key is in. heads_first:
    [pages, hk, page, d] in memory."""

    def __init__(self, lens, hk, d, page, seed=1, fill=0.0, extra=3, heads_first=False, wide=2):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        total = sum(need) + extra
        order = torch.randperm(total, generator=g)
        self.pages = torch.full((len(lens), max(need + [0]) + wide), -9, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            self.pages[s, :n] = order[at:at + n].int()
            at += n
        self.k_len, self.page = lens, page
        shape = (total, hk, page, d) if heads_first else (total, page, hk, d)
        both = []
        for i in range(2):
            c = torch.full(shape, fill, dtype=BF)
            c = c.transpose(1, 2) if heads_first else c
            data = _randn((sum(lens), hk, d), seed + 10 + i)
            x = 0
            for s, n in enumerate(lens):
                for p in range(need[s]):
                    m = min(page, n - p * page)
                    c[self.pages[s, p].long(), :m] = data[x:x + m]
                    x += m
            both.append((c, data))
        (self.k, self.K), (self.v, self.V) = both
        self.starts = _starts(lens)

    def dev(self):
        def up(c):  # the strides too
            order = sorted(range(4), key=lambda i: -c.stride(i))
            back = [order.index(i) for i in range(4)]
            return c.permute(order).to(DEV).permute(back)
        return up(self.k), up(self.v), self.pages.to(DEV), _i32(self.k_len)


CASES = [
    ([(1, 1)], 1, 1, 8, 16), ([(1, 1)], 4, 2, 128, 64), ([(1, 300)], 32, 8, 128, 16), ([(3, 3)], 2, 1, 16, 16),
    ([(64, 64), (65, 65), (0, 0), (1, 1), (130, 130)], 8, 2, 64, 32),
    ([(5, 3), (4, 0), (0, 7), (1, 1), (0, 0)], 4, 4, 64, 16),  # rows that see no key
    ([(1, 1000), (2, 63), (1, 64), (3, 65), (1, 129)], 16, 2, 128, 16),
    ([(1, 5000), (1, 100), (1, 4097), (2, 1)], 8, 2, 128, 64),  # keys cut into pieces
    ([(7, 3000)], 4, 1, 72, 256), ([(300, 300)], 3, 3, 80, 16), ([(200, 1000)], 7, 1, 128, 16),
    ([(33, 33)] * 5, 6, 3, 40, 16), ([(1025, 1025)], 2, 1, 96, 1024), ([(17, 9), (9, 17)], 9, 3, 24, 16),
    ([(1, 2)] * 70 + [(2, 5)] * 70, 4, 2, 32, 16), ([(40, 20000)], 2, 2, 120, 128),
    ([(1, 700)] * 20 + [(400, 400)] + [(1, 90)] * 43, 2, 2, 64, 16),  # a prompt among single tokens
    ([(1, 33)] * 9 + [(3, 9000)] + [(0, 50)] * 3, 8, 2, 128, 32),
    ([(1, 100)] * 31 + [(1, 20000)] + [(1, 1)] * 32, 16, 2, 128, 16),  # one long among short
    ([(600, 700), (1, 1), (1, 5000), (50, 6000)], 4, 1, 80, 64),
    ([(1, 40)], 64, 1, 64, 16), ([(2, 3000), (1, 9)], 33, 1, 64, 32),  # groups past the few rows
    ([(100, 150)] + [(0, 5)] * 60 + [(1, 40)] * 20, 4, 2, 64, 16),  # few rows on average only
    ([(0, 9)] * 50 + [(70, 6000)] + [(1, 2000)] * 30, 4, 1, 128, 32),
    ([(33, 40)] * 70, 2, 1, 64, 16), ([(40, 900), (3, 2500)] * 40, 2, 2, 72, 64)]  # more than 64 longer ones


@pytest.mark.parametrize("lens,hq,hk,d,page", CASES)
@pytest.mark.parametrize("causal", [True, False])
def test_paged_attention_matches_definition(lens, hq, hk, d, page, causal):
    print(f"[case] paged {lens[:5]} hq={hq} hk={hk} d={d} page={page} causal={causal}", flush=True)
    qs = _starts([a for a, _ in lens])
    c = Cache([b for _, b in lens], hk, d, page, fill=float("nan"), heads_first=hq % 2 == 0)
    Q = _randn((qs[-1], hq, d), 1, 2.0)
    got = L.paged_attention(Q.to(DEV), *c.dev(), _i32(qs), causal=causal)
    _check(got, Q, c.K, c.V, qs, c.starts, causal)


@pytest.mark.parametrize("d", list(range(8, 129, 8)))
@pytest.mark.parametrize("lens", [[(70, 70), (0, 5), (40, 150)], [(1, 75), (2, 2)]])
def test_paged_attention_every_head_size(lens, d):
    print(f"[case] paged lens={lens} d={d}", flush=True)
    qs = _starts([a for a, _ in lens])
    c = Cache([b for _, b in lens], 2, d, 16, seed=d)
    Q = _randn((qs[-1], 6, d), d)
    _check(L.paged_attention(Q.to(DEV), *c.dev(), _i32(qs)), Q, c.K, c.V, qs, c.starts)


@pytest.mark.parametrize("each,lens,hq", [(1, [1, 50, 3000, 17], 8), (3, [3, 50, 2, 170], 4),
                                          (40, [40, 500], 2), (200, [100, 1500, 200], 2)])
def test_paged_attention_without_starts_and_shared_pages(each, lens, hq):
    """Even rows; all sequences after the first have the first page of the first."""
    print(f"[case] paged even {each} {lens}", flush=True)
    c = Cache(lens, 2, 64, 16)
    c.pages[1:, 0] = c.pages[0, 0]
    Kc, ks = O.paged_keys(c.k, c.pages, lens)
    Vc, _ = O.paged_keys(c.v, c.pages, lens)
    K, V = torch.from_numpy(Kc).to(BF), torch.from_numpy(Vc).to(BF)
    qs = [each * i for i in range(len(lens) + 1)]
    Q = _randn((qs[-1], hq, 64), 5)
    _check(L.paged_attention(Q.to(DEV), *c.dev()), Q, K, V, qs, ks)
    _check(L.paged_attention(Q.to(DEV), *c.dev(), _i32(qs), scale=0.3), Q, K, V, qs, ks, scale=0.3)


@pytest.mark.parametrize("lens", [[(40, 40), (25, 25)], [(1, 9000), (1, 8500)]])
def test_paged_attention_strides_and_rows_of_no_sequence(lens):
    print(f"[case] paged strides {lens}", flush=True)
    hq, hk, d, front, back = 8, 4, 80, 3, 5
    qs = [front + v for v in _starts([a for a, _ in lens])]
    c = Cache([b for _, b in lens], hk, d, 16)
    k, v, pages, k_len = c.dev()
    wide = torch.zeros(*k.shape[:2], hk + 1, 2 * d + 16, dtype=BF, device=DEV)
    wide[:, :, 1:, 8:8 + d], wide[:, :, 1:, 8 + d:8 + 2 * d] = k, v
    nq = qs[-1] + back
    qall = _randn((nq, hq + 6, d + 16), 10)
    buf = torch.full((nq, hq + 1, d + 8), 9.0, dtype=BF, device=DEV)
    out = buf[:, :hq, 8:]
    got = L.paged_attention(qall.to(DEV)[:, 2:2 + hq, 8:8 + d], wide[:, :, 1:, 8:8 + d],
                            wide[:, :, 1:, 8 + d:8 + 2 * d], pages, k_len, _i32(qs), O=out)
    assert got is out
    _check(got, qall[:, 2:2 + hq, 8:8 + d], c.K, c.V, qs, c.starts)
    out[front:nq - back] = 9.0
    assert torch.all(buf == 9.0)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("lens", [[(70, 70), (90, 90)], [(3, 5000), (2, 4000)]])
def test_paged_attention_hidden_keys_never_enter(lens, value):
    print(f"[case] paged hidden non-finite {lens} {value}", flush=True)
    hq, hk, d = 4, 2, 64
    qs = _starts([a for a, _ in lens])
    c = Cache([b for _, b in lens], hk, d, 32, fill=value)
    n0 = c.k_len[0]
    # the first sequence's last keys are seen by its last queries only
    for key, cache, packed, h, e, x in ((n0 - 1, c.v, c.V, 0, 5, value), (n0 - 1, c.v, c.V, 1, 7, float("nan")),
                                        (n0 - 2, c.k, c.K, 1, slice(None), float("nan"))):
        cache[c.pages[0, key // 32].long(), key % 32, h, e] = x
        packed[key, h, e] = x
    Q = _randn((qs[-1], hq, d), 12)
    got = L.paged_attention(Q.to(DEV), *c.dev(), _i32(qs))
    _check(got, Q, c.K, c.V, qs, c.starts)
    g = got.float().cpu()
    assert torch.all(g[:qs[1] - 2].isfinite()) and torch.all(g[qs[1]:].isfinite())


def test_paged_attention_lengths_pages_and_starts_out_of_range():
    """Lengths and starts are moved to the ends, pages outside the pool to its ends; starts that
    do not ascend stay inside the tensors; no pages at all give zeros."""
    print("[case] paged out of range", flush=True)
    c = Cache([100, 200], 2, 64, 16, extra=0, wide=0)
    Q = _randn((40, 4, 64), 19)
    k, v, pages, k_len = c.dev()
    far = _i32([2 ** 31 - 1, -5])
    full = pages[:1].expand(2, -1).contiguous()
    width = pages.shape[1] * 16
    Kc, _ = O.paged_keys(c.k, full.cpu().clamp(0, k.shape[0] - 1), [width, 0])
    Vc, _ = O.paged_keys(c.v, full.cpu().clamp(0, k.shape[0] - 1), [width, 0])
    got = L.paged_attention(Q.to(DEV), k, v, full, far, _i32([-7, 25, 1000]))
    _check(got, Q, torch.from_numpy(Kc).to(BF), torch.from_numpy(Vc).to(BF), [0, 25, 40], [0, width, width])
    bad = pages.clone()
    bad[0, :3] = torch.tensor([-2 ** 31, 2 ** 31 - 1, k.shape[0]], dtype=torch.int32)
    ends = bad.cpu().clamp(0, k.shape[0] - 1)
    Kc, ks = O.paged_keys(c.k, ends, [100, 200])
    Vc, _ = O.paged_keys(c.v, ends, [100, 200])
    got = L.paged_attention(Q.to(DEV), k, v, bad, k_len, _i32([0, 15, 40]))
    _check(got, Q, torch.from_numpy(Kc).to(BF), torch.from_numpy(Vc).to(BF), [0, 15, 40], ks)
    buf = torch.full((60, 4, 64), 9.0, dtype=BF, device=DEV)
    many = pages[[0, 1, 0, 1]].contiguous()
    L.paged_attention(Q.to(DEV), k, v, many, _i32([100, 200, 50, 7]),
                      _i32([30, 2 ** 31 - 1, 5, -2 ** 31, 38]), O=buf[10:50])
    # the same rows asked for again and again
    big = _randn((400, 4, 64), 20).to(DEV)
    L.paged_attention(big, k, v, pages[[0, 1] * 40].contiguous(), k_len.repeat(40),
                      _i32([0, 400] * 40 + [0]))
    L.paged_attention(Q.to(DEV), k, v, pages[[0, 1] * 40].contiguous(), k_len.repeat(40),
                      _i32([0, 5] * 40 + [0]))
    torch.cuda.synchronize()
    assert torch.all(buf[:10] == 9.0) and torch.all(buf[50:] == 9.0)
    assert torch.all(L.paged_attention(Q.to(DEV), k, v, pages[:, :0], k_len, _i32([0, 15, 40])) == 0)
    assert torch.all(L.paged_attention(Q.to(DEV), k[:0], v[:0], pages, k_len, _i32([0, 15, 40])) == 0)
    assert L.paged_attention(Q.to(DEV)[:0], k, v, pages, k_len).shape == (0, 4, 64)


@pytest.mark.parametrize("lens", [[(130, 130), (1, 70)], [(1, 7000), (1, 100)], [(90, 5000), (1, 3000)]])
def test_paged_attention_repeats_without_workspace_and_on_streams(lens):
    print(f"[case] paged repeats {lens}", flush=True)
    qs = _starts([a for a, _ in lens])
    c = Cache([b for _, b in lens], 2, 128, 16)
    Q = _randn((qs[-1], 8, 128), 22)
    d, qd, qsd = c.dev(), Q.to(DEV), _i32(qs)
    first = L.paged_attention(qd, *d, qsd)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            outs += [L.paged_attention(qd, *d, qsd) for _ in range(2)]
    for st in streams:
        st.synchronize()
    assert all(torch.equal(first, o) for o in outs)
    out = torch.empty_like(first)
    cache = L._paged_cache(0, *d)
    p = L.PagedParams(qs[-1], 8, 1024, 128, 1024, 128, 1, 0, 128 ** -0.5)
    assert L.lib().th_paged_attention(L._ptr(qd), L.TH_BF16, L._ptr(qsd), cache, p, L._ptr(out), None, 0,
                                      L._stream()) == L.TH_OK
    _check(out, Q, c.K, c.V, qs, c.starts)


def test_paged_store_and_attention_captured_and_replayed_with_new_lengths():
    """Single tokens in two graphs that share a workspace: keys are stored and attended to,
    lengths and pages change between replays, eager work runs between them."""
    print("[case] paged in a graph", flush=True)
    nseq, hq, hk, d, page = 3, 8, 2, 128, 16
    c = Cache([4000, 4000, 4000], hk, d, page)
    k, v, pages, k_len = c.dev()
    Q, new = _randn((nseq, hq, d), 25).to(DEV), _randn((nseq, 2 * hk, d), 26).to(DEV)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)

    def step():
        L.cache_store(new[:, :hk], new[:, hk:], k, v, pages, k_len)
        return L.paged_attention(Q, k, v, pages, k_len, ws=ws)

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for i, lens in enumerate(([1, 2, 3], [4000, 1, 3999], [64, 65, 4000], [640, 17, 1])):
        k_len.copy_(_i32(lens))
        pages.copy_(c.pages[[i % 3, (i + 1) % 3, (i + 2) % 3]])
        Q.copy_(_randn((nseq, hq, d), 30 + i))
        new.copy_(_randn((nseq, 2 * hk, d), 40 + i))
        graphs[i % 2].replay()
        eager = step()
        torch.cuda.synchronize()
        assert torch.equal(outs[i % 2], eager)
        Kc, ks = O.paged_keys(k.cpu(), pages.cpu(), lens)
        Vc, _ = O.paged_keys(v.cpu(), pages.cpu(), lens)
        assert np.array_equal(Kc[np.array(ks[1:]) - 1], new[:, :hk].cpu().double().numpy())
        _check(eager, Q.cpu(), torch.from_numpy(Kc).to(BF), torch.from_numpy(Vc).to(BF), [0, 1, 2, 3], ks)


def test_paged_cache_past_32_bits():
    print("[case] paged keys past 2^32 elements", flush=True)
    pages, page, d = 40, 16, 64
    pitch = (1 << 23) + 8  # of a token: a page is past 2^27 elements, the cache past 2^32
    buf = torch.empty(pages * page * pitch + 2 * d, dtype=BF, device=DEV)
    k = buf.as_strided((pages, page, 1, d), (page * pitch, pitch, d, 1))
    v = buf.as_strided((pages, page, 1, d), (page * pitch, pitch, d, 1), d)
    n = pages * page - 5
    K, V, Q = _randn((n, 1, d), 31), _randn((n, 1, d), 32), _randn((5, 3, d), 33)
    table, k_len = torch.randperm(pages).int()[None].to(DEV), _i32([n])
    L.cache_store(K.to(DEV), V.to(DEV), k, v, table, k_len)
    _check(L.paged_attention(Q.to(DEV), k, v, table, k_len), Q, K, V, [0, 5], [0, n])
    Q = _randn((50, 3, d), 34)
    _check(L.paged_attention(Q.to(DEV), k, v, table, k_len), Q, K, V, [0, 50], [0, n])


@pytest.mark.parametrize("lens,hk,d,page", [
    ([(1, 1)], 1, 8, 16), ([(1, 50), (1, 33), (1, 16), (1, 17)], 8, 128, 16), ([(70, 70), (0, 9), (40, 150)], 2, 64, 32),
    ([(5, 3), (4, 0), (2, 2)], 3, 24, 16), ([(1, 5)] * 150, 1, 72, 16), ([(300, 1000), (1, 1)], 32, 128, 64)])
@pytest.mark.parametrize("heads_first", [True, False])
def test_store_matches_definition(lens, hk, d, page, heads_first):
    """Rows before the first key of their sequence, and all other places of the pool, stay."""
    print(f"[case] store {lens[:4]} hk={hk} d={d} page={page} {heads_first}", flush=True)
    front, back = 2, 3
    qs = [front + x for x in _starts([a for a, _ in lens])]
    c = Cache([b for _, b in lens], hk, d, page, fill=9.0, heads_first=heads_first)
    kv = _randn((qs[-1] + back, 2 * hk + 1, d + 8), 5)
    K, V = kv[:, :hk, :d], kv[:, hk:2 * hk, 8:]
    k, v, pages, k_len = c.dev()
    dv = kv.to(DEV)
    L.cache_store(dv[:, :hk, :d], dv[:, hk:2 * hk, 8:], k, v, pages, k_len, _i32(qs))
    for got, old, new in ((k, c.k, K), (v, c.v, V)):
        want = O.paged_store(old, new, c.pages.tolist(), c.k_len, qs)
        assert np.array_equal(got.double().cpu().numpy(), want)


def test_store_out_of_range():
    """Pages outside the pool are not written, nor is any other memory; even rows."""
    print("[case] store out of range", flush=True)
    hk, d, page = 2, 64, 16
    pool = torch.full((12, page, hk, d), 9.0, dtype=BF, device=DEV)
    k, v = pool[1:5], pool[7:11]
    pages = _i32([0, -1, 4, 3, 2 ** 31 - 1, 1]).view(2, 3)
    K, V = _randn((6, hk, d), 1), _randn((6, hk, d), 2)
    for lens, qs in (([48, 20], None), ([2 ** 31 - 1, -4], None), ([1, 18], None),
                     ([17, 48], [-3, 2, 900]), ([40, 48], [5, 1, 3])):
        pool.fill_(9.0)
        L.cache_store(K.to(DEV), V.to(DEV), k, v, pages, _i32(lens), None if qs is None else _i32(qs))
        assert torch.all(pool[[0, 5, 6, 11]] == 9.0)
        if qs != [5, 1, 3]:
            q = [0, 3, 6] if qs is None else [min(max(x, 0), 6) for x in qs]
            n = [min(max(x, 0), 48) for x in lens]
            for got, new in ((k, K), (v, V)):
                want = O.paged_store(np.full(tuple(k.shape), 9.0), new, pages.tolist(), n, q)
                assert np.array_equal(got.double().cpu().numpy(), want)
    pool.fill_(9.0)
    L.cache_store(K.to(DEV), V.to(DEV), k[:0], v[:0], pages, _i32([5, 5]))
    L.cache_store(K.to(DEV)[:0], V.to(DEV)[:0], k, v, pages, _i32([5, 5]))
    L.cache_store(K.to(DEV), V.to(DEV), k, v, pages[:, :0], _i32([5, 5]))
    assert torch.all(pool == 9.0)
