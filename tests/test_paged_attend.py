"""gsa_paged_attend and gsa_paged_unfold (raw rows in 8 bits in a paged cache)
against plain 64-bit attention over the values that the codes stand for."""
import math

import pytest
import torch

from _paged import Cache, logit_error, lse_tolerance, softmax_av, tolerance

pytestmark = pytest.mark.gpu

G = None
LOG2E = math.log2(math.e)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    global G
    from long_context_gsa_b200 import build
    build.build_library()
    import long_context_gsa_b200 as G_
    G = G_


def code_of(name):
    return {"bf16": G.GSA_BF16, "f32": G.GSA_F32, "i8": G.GSA_I8, "e4m3": G.GSA_E4M3}[name]


def descs(c, hq, *, dtype="bf16", out="f32", topk=0, n_max=1, exclude=True, scale=0.0):
    desc = G.make_desc(len(c.lens), hq, c.hkv, c.d, c.chunk, n_max, c.cap, topk, exclude, scale, code_of(dtype),
                       code_of(out))
    pdesc = G.make_pdesc(code_of(c.fmt), c.page, c.n_pages, c.max_pages)
    ws = torch.empty(G.gsa_workspace_bytes(desc, G.GSA_OP_PAGED), dtype=torch.uint8, device="cuda")
    G.gsa_workspace_init(ws)
    return desc, pdesc, ws


def check_row(got, got_lse, q, k, v, z_extra, v_extra, scale, d, out_bf16, what, prior=False):
    """One output row against exact attention of q over rows k, v and the given extra logits and values."""
    z = (k @ q) * scale
    dz = 0.0
    if len(k):
        reach = float((k.abs() @ q.abs()).max()) * scale * LOG2E
        dz = logit_error(d, reach, float(q.abs().max() * k.abs().sum(-1).max()) * scale * LOG2E)
    vv = v
    if z_extra is not None:
        z, vv = torch.cat([z, z_extra]), torch.cat([v, v_extra])
    ref, lse = softmax_av(z, vv)
    vmax = float(vv.abs().max()) if len(vv) else 0.0
    err = (got.double() - ref).abs()
    lim = tolerance(dz, vmax, out_bf16, ref, prior)
    allowed = float(torch.as_tensor(lim).max())
    assert bool((err <= lim).all()), f"{what}: off by {float(err.max()):.3e}, allowed {allowed:.3e}"
    if math.isinf(float(lse)):
        assert float(got_lse) == float(lse), f"{what}: lse {float(got_lse)}"
    else:
        assert abs(float(got_lse) - float(lse)) <= lse_tolerance(dz, float(lse)), f"{what}: lse"


def run_attend(c, hq, n_q, *, dtype="bf16", out="f32", seed=1, scale=0.0, n_gists=None, own_len=None, q_std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    desc, pdesc, ws = descs(c, hq, dtype=dtype, out=out, scale=scale, n_max=max(1, c.cap // c.chunk))
    B = len(c.lens)
    q = (torch.randn((B, n_q, hq, c.d), generator=g, device="cuda") * q_std).to(DT[dtype])
    o = torch.full((B, n_q, hq, c.d), float("nan"), dtype=DT[out], device="cuda")
    lse = torch.full((B, n_q, hq), float("nan"), device="cuda")
    own = own_len if own_len is not None else torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    G.gsa_paged_attend(desc, pdesc, n_q, q, *c.args(), n_gists, own, o, lse, ws)
    return q, o, lse, ws, (desc, pdesc, own)


def check_attend(c, hq, n_q, q, o, lse, *, out="f32", scale=0.0, skip=lambda b, r: False):
    s = scale or 1 / math.sqrt(c.d)
    G_ = hq // c.hkv
    for b, n in enumerate(c.lens):
        k, v = c.rows("k", b, n), c.rows("v", b, n)
        keep = torch.tensor([not skip(b, r) for r in range(n)], dtype=torch.bool, device="cuda")
        for i in range(n_q):
            end = max(0, n - (n_q - 1) + i)
            at = keep[:end]
            for h in range(hq):
                check_row(o[b, i, h], lse[b, i, h], q[b, i, h].double(), k[h // G_, :end][at], v[h // G_, :end][at],
                          None, None, s, c.d, out == "bf16", f"seq {b} query {i} head {h}")


EDGES = [0, 1, 15, 16, 17, 127, 128, 129, 513]
ATTEND = [
    # fmt, d, hq, hkv, chunk, page, lens, n_q, dtype, out
    ("e4m3", 64, 8, 2, 8, 64, EDGES, 1, "bf16", "f32"),
    ("i8", 64, 8, 2, 8, 64, EDGES, 1, "bf16", "bf16"),
    ("e4m3", 128, 7, 1, 16, 16, EDGES, 1, "bf16", "bf16"),
    ("i8", 128, 7, 1, 16, 128, EDGES, 1, "bf16", "f32"),
    ("i8", 128, 4, 4, 24, 24, EDGES, 1, "f32", "f32"),           # pages that end inside a tile
    ("e4m3", 64, 2, 1, 7, 7, [3, 50, 300], 1, "f32", "f32"),     # odd blocks, pages of 7 rows
    ("e4m3", 64, 1, 1, 1, 1, [1, 33, 40], 1, "f32", "bf16"),     # one row a block and a page
    ("i8", 128, 16, 1, 64, 192, [65, 700], 1, "bf16", "f32"),    # 16 query rows in one group
    ("e4m3", 128, 16, 2, 32, 64, [5, 200, 129], 3, "bf16", "f32"),   # 24 rows: causal, two groups
    ("i8", 64, 12, 4, 8, 32, [2, 16, 260], 5, "f32", "f32"),     # more queries than rows
    ("e4m3", 64, 16, 1, 16, 64, [64, 300], 64, "bf16", "bf16"),  # the most query tokens
    ("i8", 128, 4, 1, 16, 48, [3001, 90], 5, "f32", "f32"),      # causal, cut over several CTAs, 16 + 4 rows
    ("e4m3", 64, 6, 2, 8, 64, [2500], 3, "bf16", "bf16"),
]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "{}_d{}_{}x{}_c{}_p{}_q{}_{}_{}".format(*c[:6], *c[7:]))
def test_attend(case):
    fmt, d, hq, hkv, chunk, page, lens, n_q, dtype, out = case
    c = Cache(lens, hkv, d, chunk, page, fmt, seed=d + chunk + n_q)
    q, o, lse, ws, _ = run_attend(c, hq, n_q, dtype=dtype, out=out)
    check_attend(c, hq, n_q, q, o, lse, out=out)
    assert G.gsa_workspace_status(ws) == 0


@pytest.mark.parametrize("fmt,d", [("e4m3", 64), ("i8", 128)])
def test_attend_long_and_ragged_over_many_ctas(fmt, d):
    """Sequences cut over many CTAs next to short ones; repeated calls give the same bits."""
    c = Cache([70001, 1, 0, 5000, 313], 1, d, 16, 64, fmt, seed=5)
    q, o, lse, ws, (desc, pdesc, own) = run_attend(c, 4, 1)
    check_attend(c, 4, 1, q, o, lse)
    for _ in range(3):
        o2, l2 = torch.empty_like(o), torch.empty_like(lse)
        G.gsa_paged_attend(desc, pdesc, 1, q, *c.args(), None, own, o2, l2, ws)
        assert torch.equal(o2, o) and torch.equal(l2, lse)
    assert G.gsa_workspace_status(ws) == 0


def test_attend_sharp_and_huge_logits():
    """Logits of several hundred: the reference maximum moves, far weights vanish."""
    c = Cache([900], 2, 64, 8, 32, "e4m3", seed=6, std=4.0)
    q, o, lse, _, _ = run_attend(c, 8, 1, q_std=8.0)
    check_attend(c, 8, 1, q, o, lse)
    q, o, lse, _, _ = run_attend(c, 8, 1, scale=3.0)
    check_attend(c, 8, 1, q, o, lse, scale=3.0)
    # tiny and huge queries: the power-of-two scaling of a row
    for std in (1e-30, 1e-6, 1e6):
        q, o, lse, _, _ = run_attend(c, 8, 1, q_std=std, scale=0.125 / std)
        check_attend(c, 8, 1, q, o, lse, scale=0.125 / std)


def test_attend_counts_gists_and_shares_pages():
    """Lengths as n_gists * chunk + own_len, clamped to t_max; two sequences reading the same prefix pages."""
    c = Cache([200, 200, 77], 2, 64, 8, 16, "i8", seed=7, share=4)
    n = torch.tensor([24, 25, 9], dtype=torch.int32, device="cuda")
    own = torch.tensor([8, 500, 5], dtype=torch.int32, device="cuda")  # the second is cut at t_max = 200
    q, o, lse, _, _ = run_attend(c, 4, 1, n_gists=n, own_len=own)
    check_attend(c, 4, 1, q, o, lse)


def test_attend_leaves_out_bad_pages_and_flags_them():
    c = Cache([160, 100], 2, 64, 8, 16, "e4m3", seed=8)
    c2 = Cache([160, 100], 2, 64, 8, 16, "e4m3", seed=8)
    c.table[0, 2] = -1
    c.table[1, 3] = c.n_pages
    c.table[1, 8] = 1 << 30  # past the sequence's rows: never read
    q, o, lse, ws, _ = run_attend(c, 4, 1)
    check_attend(c2, 4, 1, q, o, lse, skip=lambda b, r: r // 16 == (2 if b == 0 else 3))
    assert G.gsa_workspace_status(ws) == G.GSA_DEVERR_BAD_INDEX


def test_attend_nan_block_reaches_only_the_rows_that_see_it():
    c = Cache([64, 64], 1, 64, 8, 16, "i8", seed=9)
    clean = Cache([64, 64], 1, 64, 8, 16, "i8", seed=9)
    pid = int(c.table[0, 3])
    for kv in "kv":  # rows 56..63 of sequence 0
        c.scales[kv][pid, 0, 1] = float("nan")
    q, o, lse, _, _ = run_attend(c, 2, 8)
    # query i sees rows 0 .. 56 + i: all of them see row 56
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
    q, o, lse, _, _ = run_attend(c, 2, 12)
    assert torch.isnan(o[0, 4:]).all() and torch.isfinite(o[0, :4]).all()  # queries 0..3 end before row 56
    q2, o2, lse2, _, _ = run_attend(clean, 2, 12)
    assert torch.equal(q, q2) and torch.equal(o[1], o2[1]) and torch.equal(lse[0, :4], lse2[0, :4])
    k, v = clean.rows("k", 0, 64)[0], clean.rows("v", 0, 64)[0]
    for i in range(4):
        for h in range(2):
            check_row(o[0, i, h], lse[0, i, h], q[0, i, h].double(), k[:53 + i], v[:53 + i], None, None, 1 / 8, 64,
                      False, f"query {i} head {h}")


def test_attend_on_another_stream_and_replayed():
    c = Cache([300, 41], 2, 128, 16, 32, "e4m3", seed=10)
    q, o, lse, ws, (desc, pdesc, own) = run_attend(c, 8, 1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, l2 = torch.zeros_like(o), torch.zeros_like(lse)
    with torch.cuda.stream(side):
        G.gsa_paged_attend(desc, pdesc, 1, q, *c.args(), None, own, o2, l2, ws)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        G.gsa_paged_attend(desc, pdesc, 1, q, *c.args(), None, own, o2, l2, ws)
    for n in ([300, 41], [17, 0], [1, 30]):  # lengths change between replays
        own.copy_(torch.tensor(n, dtype=torch.int32))
        o2.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        c.lens = n
        check_attend(c, 8, 1, q, o2, l2)


def test_pool_beyond_4_gb():
    """Pages whose bytes lie past 2^32 (and whose rows times 128 do): attention, unfolding and an append there."""
    small = Cache([700], 8, 128, 16, 64, "i8", seed=30)
    total = (5 << 30) // (8 * 64 * 128)
    first = total - small.n_pages
    big = Cache.__new__(Cache)
    big.__dict__.update(small.__dict__)
    big.n_pages, big.table = total, (small.table + first).contiguous()
    big.pages, big.scales = {}, {}
    for kv in "kv":
        big.pages[kv] = torch.zeros((total, 8, 64, 128), dtype=torch.int8, device="cuda")
        big.scales[kv] = torch.zeros((total, 8, 4), device="cuda")
        big.pages[kv][first:] = small.pages[kv]
        big.scales[kv][first:] = small.scales[kv]
    q, o, lse, ws, (desc, _, own) = run_attend(big, 8, 1)
    check_attend(big, 8, 1, q, o, lse)
    x, o, lse, _ = run_unfold(big, 8, 9)
    check_unfold(big, 8, 9, x, o, lse)
    k = torch.randn((16, 8, 128), device="cuda").to(torch.bfloat16)
    at = torch.full((1,), 640, dtype=torch.int32, device="cuda")  # block 40
    pdesc = G.make_pdesc(G.GSA_I8, 64, total, big.max_pages)
    G.gsa_paged_append(desc, pdesc, G.make_append_desc(16), None, k, k, None, None, None, big.table, None, at,
                       *big.args()[:4], None, ws)
    for kv in "kv":
        got, s = big.rows(kv, 0, 656)[:, 640:], big.scales[kv][int(big.table[0, 10]), :, 0].double()[:, None, None]
        assert bool(((got - k.transpose(0, 1).double()).abs() <= 0.5 * s * (1 + 2.0 ** -10)).all())
        assert int(big.pages[kv][:first].count_nonzero()) == 0
    assert G.gsa_workspace_status(ws) == 0


def test_calls_from_two_threads():
    """Two host threads with their own streams and workspaces, batches of different sizes (different amounts of shared
    memory of the same kernel): every call succeeds and gives the bits of the same call alone."""
    import threading
    jobs = []
    for lens, seed in (([130, 7], 21), ([(13 * i) % 40 for i in range(2500)], 22)):
        c = Cache(lens, 1, 64, 8, 40, "e4m3", seed=seed)
        q, o, lse, ws, (desc, pdesc, own) = run_attend(c, 2, 1, seed=seed)
        jobs.append((c, q, o, lse, ws, desc, pdesc, own))
    torch.cuda.synchronize()
    bad = []

    def work(job):
        c, q, o, lse, ws, desc, pdesc, own = job
        stream = torch.cuda.Stream()
        try:
            with torch.cuda.stream(stream):
                for _ in range(200):
                    o2, l2 = torch.zeros_like(o), torch.zeros_like(lse)
                    G.gsa_paged_attend(desc, pdesc, 1, q, *c.args(), None, own, o2, l2, ws)
                stream.synchronize()
            if not (torch.equal(o, o2) and torch.equal(lse, l2)):
                bad.append("other bits")
        except Exception as e:  # reported by the test's own thread
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


# ------------------------------------------------------------------ unfold
def run_unfold(c, hq, topk, *, dtype="bf16", out="f32", exclude=True, seed=2, sel=None, n_gists=None, prior=None):
    """n_gists: completed chunks of each sequence (the rest of its rows are the own chunk's)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, d, hkv, chunk = len(c.lens), c.d, c.hkv, c.chunk
    N = n_gists or [n // chunk for n in c.lens]
    n_max = max(1, max(N))
    desc, pdesc, ws = descs(c, hq, dtype=dtype, out=out, topk=topk, n_max=n_max, exclude=exclude)
    x = dict(q=torch.randn((B, hq, d), generator=g, device="cuda").to(DT[dtype]),
             gist_k=torch.randn((B, hkv, n_max, d), generator=g, device="cuda").to(DT[dtype]),
             gist_v=torch.randn((B, hkv, n_max, d), generator=g, device="cuda").to(DT[dtype]),
             n=torch.tensor(N, dtype=torch.int32, device="cuda"),
             own=torch.tensor([a - b * chunk for a, b in zip(c.lens, N)], dtype=torch.int32, device="cuda"))
    if sel is None:
        sel = torch.full((B, hq, max(topk, 1)), -1, dtype=torch.int32)
        for b in range(B):
            for h in range(hq):
                cpu = torch.Generator().manual_seed(seed + 131 * b + h)
                m = torch.randperm(N[b], generator=cpu)[:topk].sort().values
                sel[b, h, :len(m)] = m
    x["sel"] = sel.cuda()
    x["score"] = torch.where(x["sel"] >= 0, torch.randn(sel.shape, generator=g, device="cuda") * 2, -math.inf)
    o = torch.full((B, hq, d), float("nan"), dtype=DT[out], device="cuda")
    lse = torch.full((B, hq), float("nan"), device="cuda")
    if not exclude:
        scores = torch.empty((B, hq, n_max), device="cuda")
        G.gsa_score_gists(desc, x["q"], x["gist_k"], x["gist_v"], x["n"], scores, ws)
    G.gsa_paged_unfold(desc, pdesc, x["q"], *c.args(), x["gist_v"], x["n"], x["own"], x["sel"] if topk else None,
                       x["score"] if topk else None, G.GSA_PRIOR_NONE if exclude else G.GSA_PRIOR_GISTS, o, lse, ws)
    return x, o, lse, ws


def check_unfold(c, hq, topk, x, o, lse, *, out="f32", exclude=True):
    G_, s = hq // c.hkv, 1 / math.sqrt(c.d)
    for b, n in enumerate(c.lens):
        N = int(x["n"][b])
        k, v = c.rows("k", b, n), c.rows("v", b, n)
        for h in range(hq):
            kv, q = h // G_, x["q"][b, h].double()
            ids = [m for m in x["sel"][b, h].tolist() if 0 <= m < N] if topk else []
            at = torch.tensor([r for m in ids for r in range(m * c.chunk, (m + 1) * c.chunk)]
                              + list(range(N * c.chunk, n)), dtype=torch.long, device="cuda")
            if exclude:
                pick = torch.tensor([i for i, m in enumerate(x["sel"][b, h].tolist()) if 0 <= m < N], device="cuda",
                                    dtype=torch.long)
                z = x["score"][b, h, pick].double() if topk else torch.zeros(0, dtype=torch.float64, device="cuda")
                gv = x["gist_v"][b, kv, torch.tensor(ids, dtype=torch.long, device="cuda")].double()
                kk, vv = k[kv, at], v[kv, at]
            else:  # every gist is attended, its key exact in the logits
                z = None
                gv = None
                kk = torch.cat([k[kv, at], x["gist_k"][b, kv, :N].double()])
                vv = torch.cat([v[kv, at], x["gist_v"][b, kv, :N].double()])
            check_row(o[b, h], lse[b, h], q, kk, vv, z, gv, s, c.d, out == "bf16", f"seq {b} head {h}",
                      prior=not exclude)


UNFOLD = [
    # fmt, d, hq, hkv, chunk, page, lens, topk, dtype, out, exclude
    ("e4m3", 64, 8, 2, 8, 64, [8 * 90 + 3, 8 * 5, 7, 0], 16, "bf16", "f32", True),
    ("i8", 64, 8, 2, 8, 64, [8 * 90 + 3, 8 * 5, 9], 16, "bf16", "bf16", False),
    ("i8", 128, 7, 1, 16, 48, [16 * 40 + 15, 16 * 3 + 1], 33, "bf16", "f32", True),
    ("e4m3", 128, 4, 1, 32, 32, [32 * 70, 32 * 8 + 31], 64, "bf16", "f32", False),
    ("i8", 64, 1, 1, 16, 64, [16 * 256 + 3], 8, "f32", "f32", True),
    ("e4m3", 128, 6, 2, 7, 21, [7 * 60 + 6, 7 * 2], 20, "f32", "f32", True),
    ("i8", 64, 4, 2, 1, 3, [40, 2], 9, "f32", "bf16", True),
    ("e4m3", 64, 4, 4, 64, 64, [64 * 20 + 63], 5, "bf16", "bf16", True),
    ("e4m3", 128, 2, 1, 16, 16, [16 * 30 + 4], 0, "bf16", "f32", False),   # no selection: gists and the own chunk
    ("i8", 64, 2, 1, 4, 256, [4 * 1100], 1024, "bf16", "f32", True),       # the most chunks
]


@pytest.mark.parametrize("case", UNFOLD, ids=lambda c: "{}_d{}_{}x{}_c{}_p{}_k{}_{}_{}_x{:d}".format(*c[:6], *c[7:]))
def test_unfold(case):
    fmt, d, hq, hkv, chunk, page, lens, topk, dtype, out, exclude = case
    c = Cache(lens, hkv, d, chunk, page, fmt, seed=chunk + topk)
    x, o, lse, ws = run_unfold(c, hq, topk, dtype=dtype, out=out, exclude=exclude)
    check_unfold(c, hq, topk, x, o, lse, out=out, exclude=exclude)
    assert G.gsa_workspace_status(ws) == 0


DECODE = [
    # fmt, dtype, d, hq, hkv, chunk, lens, topk, exclude
    ("e4m3", "bf16", 64, 8, 2, 8, [8 * 60 + 3, 8 * 9], 7, True),
    ("i8", "f32", 128, 4, 1, 16, [16 * 40 + 5], 6, True),
    ("i8", "bf16", 128, 7, 1, 16, [16 * 40 + 5, 16 * 3], 0, False),  # no selection: the gists and the own chunk
    ("e4m3", "bf16", 64, 4, 1, 1, [4200], 9, False),                 # rows too long for the selection in the scoring
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "{}_{}_d{}_{}x{}_c{}_k{}_x{:d}".format(*c[:6], *c[7:]))
def test_decode(case):
    """Score, select and unfold in one call, with and without the outputs that may be left out."""
    fmt, dtype, d, hq, hkv, chunk, lens, topk, exclude = case
    c = Cache(lens, hkv, d, chunk, 2 * chunk, fmt, seed=topk + 40)
    N = [n // chunk for n in lens]
    g = torch.Generator(device="cuda").manual_seed(41)
    desc, pdesc, ws = descs(c, hq, dtype=dtype, topk=topk, n_max=max(N), exclude=exclude)
    B = len(lens)
    q, gk, gv = (torch.randn(s, generator=g, device="cuda").to(DT[dtype]) for s in
                 ((B, hq, d), (B, hkv, max(N), d), (B, hkv, max(N), d)))
    n = torch.tensor(N, dtype=torch.int32, device="cuda")
    own = torch.tensor([a - b * chunk for a, b in zip(lens, N)], dtype=torch.int32, device="cuda")
    o, lse, o2 = (torch.empty(s, device="cuda") for s in ((B, hq, d), (B, hq), (B, hq, d)))
    sel = torch.full((B, hq, max(topk, 1)), -1, dtype=torch.int32, device="cuda")
    score = torch.empty((B, hq, max(topk, 1)), device="cuda")
    G.gsa_paged_decode(desc, pdesc, q, gk, gv, *c.args(), n, own, o, lse, sel if topk else None,
                       score if topk else None, ws)
    G.gsa_paged_decode(desc, pdesc, q, gk, gv, *c.args(), n, own, o2, None, None, None, ws)
    assert torch.equal(o, o2) and G.gsa_workspace_status(ws) == 0
    # the selection is the top of the scores, up to scores that fp32 cannot tell apart
    for b in range(B):
        for h in range(hq):
            z = gk[b, h // (hq // hkv), :N[b]].double() @ q[b, h].double() / math.sqrt(d)
            got = [m for m in sel[b, h].tolist() if m >= 0]
            assert len(got) == min(topk, N[b]) == len(set(got))
            if got:
                kth = float(z.topk(len(got)).values.min())
                assert all(float(z[m]) >= kth - 1e-5 * max(1.0, abs(kth)) for m in got)
    check_unfold(c, hq, topk, dict(q=q, gist_k=gk, gist_v=gv, n=n, sel=sel, score=score), o, lse, exclude=exclude)


def test_unfold_own_chunk_full_and_bad_entries():
    """A full own chunk (before its gist step); -1 between entries, entries >= N skipped and flagged, unsorted lists."""
    c = Cache([8 * 21, 8 * 10 + 8], 1, 64, 8, 32, "e4m3", seed=11)
    sel = torch.tensor([[[5, -1, 0, 19, -1, 3]], [[9, 200, 1, -1, -1, 8]]], dtype=torch.int32)
    x, o, lse, ws = run_unfold(c, 1, 6, sel=sel, n_gists=[20, 10])
    x["score"][1, 0, 1] = -math.inf
    check_unfold(c, 1, 6, x, o, lse)
    assert G.gsa_workspace_status(ws) == G.GSA_DEVERR_BAD_INDEX


def test_unfold_bad_page_is_left_out():
    c = Cache([8 * 20], 1, 64, 8, 8, "i8", seed=12)
    sel = torch.tensor([[[2, 7, 11]]], dtype=torch.int32)
    bad = c.table.clone()
    bad[0, 7] = -5
    good = c.table
    c.table = bad
    x, o, lse, ws = run_unfold(c, 1, 3, sel=sel, n_gists=[20])
    assert G.gsa_workspace_status(ws) == G.GSA_DEVERR_BAD_INDEX
    c.table = good
    # chunk 7's rows are out; its gist (from sel_score and gist_v) stays
    q, s = x["q"][0, 0].double(), 1 / 8
    at = torch.tensor([16 + i for i in range(8)] + [88 + i for i in range(8)], device="cuda")
    k, v = c.rows("k", 0, 160)[0, at], c.rows("v", 0, 160)[0, at]
    check_row(o[0, 0], lse[0, 0], q, k, v, x["score"][0, 0].double(), x["gist_v"][0, 0, [2, 7, 11]].double(), s, 64,
              False, "bad page")


def test_unfold_nan_block_shows():
    c = Cache([8 * 12], 1, 64, 8, 16, "e4m3", seed=13)
    c.scales["v"][int(c.table[0, 1]), 0, 0] = float("nan")  # chunk 2
    sel = torch.tensor([[[1, 2], [0, 4]]], dtype=torch.int32)
    _, o, _, _ = run_unfold(c, 2, 2, sel=sel, n_gists=[12])
    assert torch.isnan(o[0, 0]).all() and torch.isfinite(o[0, 1]).all()
