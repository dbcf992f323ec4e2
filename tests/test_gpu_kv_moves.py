"""Pages and tokens of the 4-bit cache that move, and the calls together: a decoding loop with a fork and an eviction,
captured and replayed, on two streams."""
import numpy as np
import pytest

import w4a4_quantized_linear_amd as sq
from oracle import kv as Kv

from _kv_helpers import Cache, check_attention, i32

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "int4", "nvfp4"]


@pytest.fixture(scope="module")
def td():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sq.lib()
    assert sq.device_check(), "current device is not gfx950"
    return torch, torch.device("cuda:0")


@pytest.mark.parametrize("heads,page,planes,n", [(1, 16, 1, 1), (3, 32, 2, 7), (8, 128, 3, 300), (2, 16, 1, 700)])
def test_copy(td, heads, page, planes, n):
    torch, dev = td
    kv = sq.KvLayout("nvfp4", heads, 64, page)
    pages = 2 * n + 5
    g = torch.Generator(device=dev)
    g.manual_seed(n)
    pool = torch.randint(256, (planes, pages, sq.kv_page_bytes(kv)), dtype=torch.uint8, generator=g, device=dev)
    order = torch.randperm(pages, generator=g, device=dev).tolist()
    src, dst = order[:n], order[n:2 * n]
    src[-1] = src[0]                                                   # one page to two places
    want = pool.clone()
    want[:, dst] = want[:, src]
    assert sq.kv_copy(kv, pool, src, dst) is pool and torch.equal(pool, want)
    sq.kv_copy(kv, pool, [], [])
    sq.kv_copy(kv, pool, dst, dst)
    sq.kv_copy(kv, pool, np.array(src), torch.tensor(dst))
    assert torch.equal(pool, want)
    if planes == 1:
        sq.kv_copy(kv, pool[0], dst[:1], src[:1])
        assert torch.equal(pool[0, src[0]], want[0, dst[0]])


def _all_tokens(torch, dev, kv, pool, table, places):
    """K and V of every place of every sequence of one layer."""
    B = table.shape[0]
    return sq.kv_read(kv, pool, table, i32([places] * B, dev, torch), B * places,
                      cu=i32(np.arange(B + 1) * places, dev, torch), f32=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(td, fmt, D, page, in_place):
    """Kept tokens against numpy, layer by layer; every other token, also of the last tile, stays as it was."""
    torch, dev = td
    kv = sq.KvLayout(fmt, 2, D, page)
    rng = np.random.default_rng(D + page)
    lens = [1, 17, 64, 200, 333, 90]
    starts = [0, 3, 16, 5, 64, 89]
    kept = [sorted(rng.choice(np.arange(s, n), size=max(0, int(f * (n - s))), replace=False))
            for s, n, f in zip(starts, lens, (1.0, 0.5, 0.0, 0.9, 0.3, 1.0))]
    c = Cache(torch, dev, kv, lens, 11, spare=40)
    planes = 3
    pool = torch.stack([c.pool, c.pool.flip(0), c.pool])                # layer 1: other bytes, at other pages
    most = max(len(k) for k in kept) + 2
    keep = np.full((6, most), -1)
    for b, k in enumerate(kept):
        keep[b, :len(k)] = k
    before = pool.clone()
    to = c.table
    if not in_place:
        cols = max(-(-(s + len(k)) // page) for s, k in zip(starts, kept))
        tab = np.full((6, cols), -1)
        at = 0
        for b, (s, k) in enumerate(zip(starts, kept)):
            m = -(-(s + len(k)) // page)
            tab[b, :m] = c.free[at:at + m]
            at += m
        to = i32(tab, dev, torch)
    got = sq.kv_compact(kv, pool, c.table, i32(keep, dev, torch), i32([len(k) for k in kept], dev, torch),
                        start=i32(starts, dev, torch), to=None if in_place else to)
    assert got is pool
    for layer in range(planes):
        places, new_places = c.cols * page, to.shape[1] * page
        old = [t.view(6, places, -1) for t in _all_tokens(torch, dev, kv, before[layer], c.table, places)]
        was = [t.view(6, new_places, -1) for t in _all_tokens(torch, dev, kv, before[layer], to, new_places)]
        now = [t.view(6, new_places, -1) for t in _all_tokens(torch, dev, kv, pool[layer], to, new_places)]
        for o, w, x in zip(old, was, now):
            want = w.clone()
            for b, (s, k) in enumerate(zip(starts, kept)):
                if k:
                    want[b, s:s + len(k)] = o[b, torch.tensor(np.array(k), device=dev)]
            assert torch.equal(torch.nan_to_num(x, nan=-1.25), torch.nan_to_num(want, nan=-1.25)), layer
        others = torch.ones(pool.shape[1], dtype=torch.bool, device=dev)
        others[to[to >= 0].long()] = False
        assert torch.equal(pool[layer][others], before[layer][others])


@pytest.mark.parametrize("fmt", FMTS)
def test_compact_bounds(td, fmt):
    """Indexes without a place move nothing; counts beyond the list are the list's; a long sequence in place."""
    torch, dev = td
    kv = sq.KvLayout(fmt, 1, 64, 16)
    c = Cache(torch, dev, kv, [40], 12)
    before = c.pool.clone()
    for keep, n in (([[-1, -5, 48, 1 << 30]], 4), ([[3, 4, 5, 6]], 0), ([[3, 4]], -2)):
        sq.kv_compact(kv, c.pool, c.table, i32(keep, dev, torch), i32([n], dev, torch))
        assert torch.equal(c.pool, before)
    sq.kv_compact(kv, c.pool, c.table, i32([[0, 1, 2]], dev, torch), i32([99], dev, torch))
    assert torch.equal(c.pool, before)
    sq.kv_compact(kv, c.pool, c.table, i32([[5, 9]], dev, torch), i32([2], dev, torch), start=i32([200], dev, torch))
    assert torch.equal(c.pool, before)                                 # new places behind the table
    few = Cache(torch, dev, kv, [40, 90, 500], 14)                     # a wave's tiles, in two layers
    pool, keep = torch.stack([few.pool, few.pool]), np.array([[3, 5, 6] + [9] * 47, np.r_[20:70], np.r_[7:400:8]])
    sq.kv_compact(kv, pool, few.table, i32(keep, dev, torch), i32([3, 50, 50], dev, torch), start=i32([2, 15, 0], dev, torch))
    for layer in range(2):
        k, _ = sq.kv_read(kv, pool[layer], few.table, i32([40, 90, 500], dev, torch), 630, cu=i32([0, 40, 130, 630], dev, torch), f32=True)
        want = few.kh[:, 0].astype(np.float32).copy()
        want[2:5], want[40 + 15:40 + 65], want[130:180] = few.kh[keep[0, :3], 0], few.kh[40 + keep[1], 0], few.kh[130 + keep[2], 0]
        assert np.array_equal(k.cpu().numpy(), want)
    lens = [5000]
    c = Cache(torch, dev, kv, lens, 13)
    n = sq.kv_compact_bytes(kv, 1, 1, 3333)
    space = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=dev)
    keep = np.sort(c.rng.choice(5000, 3333, replace=False))
    other = c.pool.clone()
    sq.kv_compact(kv, other, c.table, i32(keep[None], dev, torch), i32([3333], dev, torch), workspace=space[256:256 + n])
    assert n > 0 and int((space[:256] != 0xA5).sum()) == 0 and int((space[256 + n:] != 0xA5).sum()) == 0
    sq.kv_compact(kv, c.pool, c.table, i32(keep[None], dev, torch), i32([3333], dev, torch))
    assert torch.equal(other, c.pool)
    k, v = sq.kv_read(kv, c.pool, c.table, i32([3333], dev, torch), 3333, cu=i32([0, 3333], dev, torch), f32=True)
    assert np.array_equal(k.cpu().numpy(), c.kh[keep, 0].astype(np.float32))
    assert np.array_equal(v.cpu().numpy(), c.vh[keep, 0].astype(np.float32))


@pytest.mark.parametrize("fmt", FMTS)
def test_decoding_loop(td, fmt):
    """Prompts, steps, a fork (full pages shared, the last one copied), drafts of which some are accepted, an
    eviction: after each the attention of the next step is the oracle's over the tokens that are left."""
    torch, dev = td
    H, Hq, D, page = 2, 8, 64, 16
    kv = sq.KvLayout(fmt, H, D, page)
    rng = np.random.default_rng(21)
    pool = torch.full((60, sq.kv_page_bytes(kv)), 255, dtype=torch.uint8, device=dev)
    free = list(rng.permutation(60))
    tab = np.full((3, 16), -1)
    lens = [0, 0, 0]
    held = [[np.zeros((0, H, D)), np.zeros((0, H, D))] for _ in range(3)]
    fake = Cache.__new__(Cache)
    fake.kv = kv
    w = Kv.F.to_bf16(1 + 0.1 * rng.standard_normal(D))
    freq = (10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
    bf = lambda x: torch.tensor(x, dtype=torch.float32).bfloat16().to(dev)

    def rows(q_lens, what, seqs=(0, 1, 2), moved=0):
        M = sum(q_lens)
        x = Kv.F.to_bf16(rng.standard_normal((M, Hq + 2 * H, D)))
        for b, q in zip(seqs, q_lens):
            lens[b] += q
            for i in range(-(-lens[b] // page)):
                if tab[b, i] < 0:
                    tab[b, i] = free.pop()
        use = list(seqs)
        t32, n32 = i32(tab[use], dev, torch), i32([lens[b] for b in use], dev, torch)
        cu = None if set(q_lens) == {1} else i32(np.r_[0, np.cumsum(q_lens)], dev, torch)
        pos = np.concatenate([lens[b] - q + np.arange(q) for b, q in zip(use, q_lens)]) + moved
        r = bf(x.reshape(M, -1))
        q = sq.kv_append(kv, pool, t32, n32, r[:, Hq * D:(Hq + H) * D], r[:, (Hq + H) * D:], cu=cu, Q=r[:, :Hq * D],
                         norm_q=bf(w), norm_k=bf(w), freq=torch.tensor(freq, device=dev), pos=i32(pos[None], dev, torch),
                         halves=True)
        kz = Kv.bf16_of(Kv.head_rows(x[:, Hq:Hq + H], w, 1e-6, freq, None, pos[None], True))
        k, v = Kv.hold(kz, fmt), Kv.hold(x[:, Hq + H:], fmt)
        at = 0
        for b, n in zip(use, q_lens):
            held[b] = [np.concatenate([held[b][0], k[at:at + n]]), np.concatenate([held[b][1], v[at:at + n]])]
            at += n
        out, lse = sq.kv_attention(kv, pool, t32, n32, q, cu=cu, lse=True)
        Qv = q.float().cpu().numpy().astype(np.float64).reshape(M, Hq, D)
        few = M * (Hq // H) <= 32 * len(use)
        check_attention(fake, Qv, out, lse, q_lens, [lens[b] for b in use], Hq, D ** -0.5, True, 0, f"{fmt} {what}",
                        "nvfp4" if fmt == "nvfp4" else "few" if few else "many", values=lambda i: tuple(held[use[i]]))

    rows([37, 90], "prompts", (0, 1))
    for i in range(3):
        rows([1, 1], f"step {i}", (0, 1))
    last = (lens[0] - 1) // page                                       # sequence 2 forks from 0
    tab[2, :last] = tab[0, :last]
    tab[2, last] = free.pop()
    sq.kv_copy(kv, pool, [int(tab[0, last])], [int(tab[2, last])])
    lens[2], held[2] = lens[0], [t.copy() for t in held[0]]
    rows([1, 1, 1], "fork")
    rows([4, 6, 5], "drafts")
    accepted = [[0, 2], [1, 3, 4, 5], []]
    start = [lens[0] - 4, lens[1] - 6, lens[2] - 5]
    keep = np.full((3, 6), -1)
    for b, a in enumerate(accepted):
        keep[b, :len(a)] = np.array(a, int) + start[b]
        held[b] = [np.concatenate([t[:start[b]], t[keep[b, :len(a)]]]) for t in held[b]]
        lens[b] = start[b] + len(a)
    sq.kv_compact(kv, pool, i32(tab, dev, torch), i32(keep, dev, torch), i32([len(a) for a in accepted], dev, torch),
                  start=i32(start, dev, torch))
    rows([1, 1, 1], "accepted", moved=7)
    stay = np.r_[0:4, 30:lens[1]]                                      # sequence 1 keeps its first tokens and the last
    fresh = np.full((1, 16), -1)
    fresh[0, :6] = [free.pop() for _ in range(6)]
    sq.kv_compact(kv, pool, i32(tab[1:2], dev, torch), i32(stay[None], dev, torch), i32([len(stay)], dev, torch),
                  to=i32(fresh, dev, torch))
    free.extend(p for p in tab[1] if p >= 0)
    tab[1], lens[1], held[1] = fresh[0], len(stay), [t[stay] for t in held[1]]
    rows([1, 1, 1], "evicted", moved=60)


def test_graph_follows_lengths(td):
    """A captured step (append, attention, workspace of its own) replayed with other lengths, rows and tables between
    eager calls, against eager results; two graphs with workspaces of their own on two streams at once."""
    torch, dev = td
    kv = sq.KvLayout("int4", 2, 128, 32)
    c = Cache(torch, dev, kv, [500, 40, 900], 31, cols=40)
    tab = c.tab.copy()
    pages = torch.full((c.pool.shape[0] + 60, c.pool.shape[1]), 255, dtype=torch.uint8, device=dev)
    pages[:c.pool.shape[0]] = c.pool
    nxt = c.pool.shape[0]
    for b in range(3):
        for i in range(40):
            if tab[b, i] < 0 and nxt < pages.shape[0]:
                tab[b, i], nxt = nxt, nxt + 1
                if i * 32 > [500, 40, 900][b] + 300:
                    break
    table, lens = i32(tab, dev, torch), i32([501, 41, 901], dev, torch)
    row = torch.randn((3, (8 + 4) * 128), device=dev).bfloat16()
    ws = [torch.empty(sq.kv_attention_bytes(kv, 40, 3, 3, 8), dtype=torch.uint8, device=dev) for _ in range(2)]

    def step(pool, w):
        q = sq.kv_append(kv, pool, table, lens, row[:, 1024:1280], row[:, 1280:], Q=row[:, :1024])
        return sq.kv_attention(kv, pool, table, lens, q, workspace=w)

    step(pages, ws[0])                                                 # every token below a length has to be there
    streams = [torch.cuda.Stream() for _ in range(2)]
    pools, graphs, outs = [pages.clone(), pages.clone()], [], []
    torch.cuda.synchronize()
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[i]):
            outs.append(step(pools[i], ws[i]))
        graphs.append(graph)
    eager = pages.clone()
    for i in range(6):
        lens += 1
        row.copy_(torch.randn_like(row))
        torch.cuda.synchronize()
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
        want = step(eager, None)
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(outs[k], want), (i, k)
            assert torch.equal(pools[k], eager), (i, k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = sq.kv_attention(kv, eager, table, lens, row[:, :1024], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, sq.kv_attention(kv, eager, table, lens, row[:, :1024]))


@pytest.mark.parametrize("fmt", FMTS)
def test_compact_walks(td, fmt):
    """In place with workgroups enough to walk: 40 sequences, 2 heads, 7 layers; the workspace form (fewer layers) on the
    same tokens gives the same bytes; and the tokens are numpy's."""
    torch, dev = td
    kv = sq.KvLayout(fmt, 2, 64, 32)
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(1, 400, 40)]
    c = Cache(torch, dev, kv, lens, 15)
    start = np.array([int(rng.integers(0, n)) for n in lens])
    kept = [np.sort(rng.choice(np.arange(s, n), int(rng.integers(0, n - s + 1)), replace=False)) for s, n in zip(start, lens)]
    keep = np.zeros((40, 400), int)
    for b, k in enumerate(kept):
        keep[b, :len(k)] = k
    args = (c.table, i32(keep, dev, torch), i32([len(k) for k in kept], dev, torch))
    many = torch.stack([c.pool] * 7)
    assert sq.kv_compact_bytes(kv, 7, 40, 400) == 0 and sq.kv_compact_bytes(kv, 1, 40, 400) > 0
    sq.kv_compact(kv, many, *args, start=i32(start, dev, torch))
    one = c.pool.clone()
    sq.kv_compact(kv, one, *args, start=i32(start, dev, torch))
    for layer in many:
        assert torch.equal(layer, one)
    M = sum(lens)
    k, v = sq.kv_read(kv, one, c.table, i32(lens, dev, torch), M, cu=i32(c.cu, dev, torch), f32=True)
    for got, held in ((k, c.kh), (v, c.vh)):
        want = held.reshape(M, -1).astype(np.float32).copy()
        for b, kk in enumerate(kept):
            want[c.cu[b] + start[b]:c.cu[b] + start[b] + len(kk)] = held.reshape(M, -1)[c.cu[b] + kk]
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_block_of_packed_layers(td, fmt):
    """A decoder's attention between packed layers: a prompt, then tokens one by one, a fork and a copy between them,
    each [Q | K | V] row from linear_w4a16 (the prompt's from linear), appended in place, attended, projected; the step as
    a captured graph with the page copy in it, replayed, against eager calls; the attention against the oracle on the
    device's own rows."""
    torch, dev = td
    H, Hq, D, page = 2, 4, 128, 16
    K, N = 512, (Hq + 2 * H) * D
    kv = sq.KvLayout(fmt, H, D, page)
    fm = "mxfp4" if fmt == "nvfp4" else fmt
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    draw = lambda *shape: torch.randn(shape, generator=g, device=dev)
    qkv, proj = sq.Layer(fm, K, N, 0), sq.Layer(fm, Hq * D, K, 0)
    pack = lambda layer: sq.pack_weight(layer, draw(layer.N, layer.K) / layer.K ** 0.5, None, None,
                                        torch.ones(layer.K, device=dev), torch.zeros(layer.N, device=dev).bfloat16())
    w_qkv, w_proj = pack(qkv), pack(proj)
    tab = np.full((2, 8), -1)
    tab[0, :6], tab[1, :6] = np.arange(6), np.arange(6, 12)
    table = i32(tab, dev, torch)
    prompt = draw(50, K).bfloat16()
    freq = (10000.0 ** (-torch.arange(64, device=dev) / 64)).float()

    def attend(pool, x, lens, cu, layer=sq.linear_w4a16):
        rows = layer(qkv, w_qkv, x, sq.EPI_BIAS)
        q, k, v = rows[:, :Hq * D], rows[:, Hq * D:(Hq + H) * D], rows[:, (Hq + H) * D:]
        sq.kv_append(kv, pool, table, lens, k, v, cu=cu, Q=q, q_out=q, freq=freq, halves=True)
        out, lse = sq.kv_attention(kv, pool, table, lens, q, cu=cu, lse=True)
        return rows, out, lse, sq.linear_w4a16(proj, w_proj, out, sq.EPI_BIAS)

    pool = torch.full((12, sq.kv_page_bytes(kv)), 255, dtype=torch.uint8, device=dev)
    attend(pool, prompt, i32([50, 0], dev, torch), i32([0, 50, 50], dev, torch), sq.linear)
    sq.kv_copy(kv, pool, [0, 1, 2, 3], [6, 7, 8, 9])                   # sequence 1 is a copy of 0
    lens, x = i32([50, 50], dev, torch), draw(2, K).bfloat16()

    def step(p):
        y = attend(p, x, lens, None)
        sq.kv_copy(kv, p, [3], [10])                                   # a page behind the sequences'
        return y

    start_pool = pool.clone()
    step(pool.clone())
    graph, held = torch.cuda.CUDAGraph(), pool.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(held)
    held.copy_(start_pool)
    for i in range(5):
        lens += 1
        x.copy_(draw(2, K).bfloat16())
        graph.replay()
        want = step(pool)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i
        assert torch.equal(pool, held), i
    n = int(lens[0])
    k, v = (t.cpu().numpy().astype(np.float64).reshape(2, n, H, D) for t in sq.kv_read(
        kv, pool, table, lens, 2 * n, cu=i32([0, n, 2 * n], dev, torch), f32=True))
    c = type("Pool", (), {})()
    c.kv, c.values = kv, lambda b: (k[b], v[b])
    c.magnitudes = lambda t: Cache.magnitudes(c, t)
    Qv = got[0][:, :Hq * D].float().cpu().numpy().astype(np.float64).reshape(2, Hq, D)
    check_attention(c, Qv, got[1], got[2], [1, 1], [n, n], Hq, D ** -0.5, True, 0, fmt, "nvfp4" if fmt == "nvfp4" else "few")
    assert torch.isfinite(got[3].float()).all()


def test_nothing_to_do(td):
    """No sequences, sequences without rows, rows without sequences, no kept tokens: nothing is read or written."""
    torch, dev = td
    kv = sq.KvLayout("int4", 2, 64, 16)
    c = Cache(torch, dev, kv, [40, 3], 1)
    was = c.pool.clone()
    none, zero = torch.zeros((0, 256), device=dev).bfloat16(), i32([0, 0, 0], dev, torch)
    lens, no_lens, no_table = i32([40, 3], dev, torch), i32([], dev, torch), c.table[:0]
    half = none[:, :128]
    for table, n, cu in ((no_table, no_lens, None), (no_table, no_lens, zero[:1]), (c.table, lens, zero)):
        assert sq.kv_append(kv, c.pool, table, n, half, half, cu=cu, Q=none).shape == (0, 256)
        assert sq.kv_attention(kv, c.pool, table, n, none, cu=cu).shape == (0, 256)
        assert sq.kv_read(kv, c.pool, table, n, 0, cu=cu)[0].shape == (0, 128)
    q, out = torch.ones((5, 256), device=dev).bfloat16(), torch.full((5, 256), 9.0, device=dev).bfloat16()
    sq.kv_attention(kv, c.pool, c.table, lens, q, cu=zero, out=out)
    sq.kv_append(kv, c.pool, c.table, lens, q[:, :128], q[:, 128:], cu=zero)
    assert (out == 9.0).all()
    sq.kv_compact(kv, c.pool, c.table, i32([[0, 1], [0, 1]], dev, torch), i32([0, -5], dev, torch))
    sq.kv_compact(kv, c.pool, c.table, i32([[], []], dev, torch), i32([7, 7], dev, torch))
    sq.kv_compact(kv, c.pool, no_table, i32(np.zeros((0, 4)), dev, torch), no_lens)
    assert torch.equal(c.pool, was)


@pytest.mark.parametrize("fmt", FMTS)
def test_pool_of_many_gigabytes(td, fmt):
    """Two layers of over 4 GiB each: the calls on pages at both ends give the bytes of the same calls on a small pool."""
    torch, dev = td
    kv = sq.KvLayout(fmt, 8, 128, 1024)
    per = sq.kv_page_bytes(kv)
    pages = (5 << 30) // per + 3
    if torch.cuda.mem_get_info()[0] < 3 * pages * per:
        pytest.skip("memory")
    big = torch.empty((2, pages, per), dtype=torch.uint8, device=dev)
    small = torch.full((2, 8, per), 255, dtype=torch.uint8, device=dev)
    where = [0, pages - 1, pages // 2, pages - 2, 1, pages - 3, pages - 4, 2]      # of the small pool's pages
    big[:, where] = small
    tab = np.array([[0, 1, 2], [3, 4, 5]])
    tables = {id(small): i32(tab, dev, torch), id(big): i32(np.array(where)[tab], dev, torch)}
    lens, cu = [3000, 2100], [0, 3000, 5100]
    g = torch.Generator(device=dev)
    g.manual_seed(2)
    x = torch.randn((5100, 2 * 1024), generator=g, device=dev).bfloat16()
    q1, q9 = (torch.randn((n, 16 * 128), generator=g, device=dev).bfloat16() for n in (2, 1800))
    keep = i32([sorted(np.random.default_rng(b).choice(2000, 900, replace=False)) for b in range(2)], dev, torch)

    def run(pool):
        table, n = tables[id(pool)], i32(lens, dev, torch)
        at = (lambda p: where[p]) if pool is big else (lambda p: p)
        for layer in pool:
            sq.kv_append(kv, layer, table, n, x[:, :1024], x[:, 1024:], cu=i32(cu, dev, torch))
        got = [sq.kv_attention(kv, layer, table, n, q1) for layer in pool]
        got.append(sq.kv_attention(kv, pool[1], table, n, q9, cu=i32([0, 900, 1800], dev, torch)))
        sq.kv_copy(kv, pool, [at(2), at(5)], [at(6), at(7)])
        sq.kv_compact(kv, pool, table, keep, i32([900, 900], dev, torch))
        to = i32([[at(2)], [at(5)]], dev, torch)
        sq.kv_compact(kv, pool, table[:, :2].contiguous(), keep[:, :100].contiguous(), i32([100, 100], dev, torch), to=to)
        return got + list(sq.kv_read(kv, pool[1], to, i32([100, 100], dev, torch), 200, cu=i32([0, 100, 200], dev, torch)))

    for a, b in zip(run(big), run(small)):
        assert torch.equal(a, b)
    assert torch.equal(big[:, where], small)
