"""Paged calls beside others: one workspace under several descriptors, several threads at once, selections of the
hierarchical calls."""
import threading

import pytest
import torch

from _paged import Cache
from test_paged_append import Pool, append, check_append
from test_paged_attend import check_unfold, code_of, descs, run_attend, run_unfold

pytestmark = pytest.mark.gpu

G = None


@pytest.fixture(scope="module", autouse=True)
def _setup():
    global G
    from long_context_gsa_b200 import build
    build.build_library()
    import long_context_gsa_b200 as G_
    import test_paged_append as P
    import test_paged_attend as A
    G = A.G = P.G = G_


def test_lengths_advance_whatever_the_workspace_served_before():
    """A dense layer (topk 0) and sparse ones (other topk) share a workspace: dense attention over cut sequences, then
    an append that advances own_len, for many values of topk."""
    B, hq, hkv, d, chunk = 4, 32, 2, 64, 8
    p = Pool(B, hkv, d, chunk, 64, 2048, "e4m3")
    dense, pdesc, _ = p.desc(hq, "bf16", n_max=64)
    sparse = {k: p.desc(hq, "bf16", n_max=64, topk=k)[0] for k in (1, 2, 3, 5, 8, 9, 10, 11, 16, 40, 64, 300)}
    ws = torch.empty(max(G.gsa_workspace_bytes(x, G.GSA_OP_PAGED) for x in [dense, *sparse.values()]),
                     dtype=torch.uint8, device="cuda")
    G.gsa_workspace_init(ws)
    own = torch.zeros(B, dtype=torch.int32, device="cuda")
    append(p, hq, own, [1900, 1500, 700, 1200], rot=64, seed=1, advance=True, state=(dense, pdesc, ws))
    assert own.tolist() == [1900, 1500, 700, 1200]
    q = torch.randn((B, 1, hq, d), device="cuda").to(torch.bfloat16)
    out, lse = torch.empty((B, 1, hq, d), device="cuda"), torch.empty((B, 1, hq), device="cuda")
    for i, (k, desc) in enumerate(sparse.items()):
        G.gsa_paged_attend(dense, pdesc, 1, q, p.pages["k"], p.pages["v"], p.scales["k"], p.scales["v"], p.table, None,
                           own, out, lse, ws)
        lens = own.tolist()
        r = append(p, hq, own, [1] * B, rot=64, seed=10 + i, advance=True, uniform=True, state=(desc, pdesc, ws))
        assert own.tolist() == [n + 1 for n in lens], f"topk {k}"
        check_append(p, r, lens, [1] * B, rounds=8)
    assert G.gsa_workspace_status(ws) == 0


def test_unfold_joins_its_rows_whatever_the_workspace_served_before():
    """The batch grows between calls on one workspace: scores of the small batch lie where the large one's rows count
    their splits."""
    hq, topk, N = 16, 60, 300
    c = Cache([8 * N + 3] * 16, 2, 64, 8, 64, "e4m3", seed=1)
    small = Cache([8 * N], 2, 64, 8, 64, "e4m3", seed=2)
    x, o, lse, _ = run_unfold(c, hq, topk)
    check_unfold(c, hq, topk, x, o, lse)
    desc, pdesc, ws = descs(c, hq, topk=topk, n_max=N)
    one = descs(small, hq, topk=topk, n_max=N)[0]
    g = torch.Generator(device="cuda").manual_seed(3)
    q, gk = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in ((1, hq, 64), (1, 2, N, 64)))
    n = torch.full((1,), N, dtype=torch.int32, device="cuda")
    own, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty((1, hq, 64), device="cuda")
    for _ in range(3):
        # the small batch's scores and selection stay in the workspace
        G.gsa_paged_decode(one, G.make_pdesc(code_of("e4m3"), 64, small.n_pages, small.max_pages), q, gk, gk,
                           *small.args(), n, own, out, None, None, None, ws)
        o2, lse2 = torch.full_like(o, float("nan")), torch.full_like(lse, float("nan"))
        G.gsa_paged_unfold(desc, pdesc, x["q"], *c.args(), x["gist_v"], x["n"], x["own"], x["sel"], x["score"],
                           G.GSA_PRIOR_NONE, o2, lse2, ws)
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
        G.gsa_workspace_init(ws)  # (the fused step of the small batch, after another one's calls)
    assert G.gsa_workspace_status(ws) == 0


def test_every_call_from_two_threads_gives_the_same_bits():
    """Two host threads begin together, each with its own stream and workspace and other amounts of shared memory; each
    of their calls is compared on its stream."""
    jobs = []
    for lens, seed in (([130, 7], 21), ([(13 * i) % 40 for i in range(2500)], 22)):
        c = Cache(lens, 1, 64, 8, 40, "e4m3", seed=seed)
        q, o, lse, ws, (desc, pdesc, own) = run_attend(c, 2, 1, seed=seed)
        jobs.append((c, q, o, lse, ws, desc, pdesc, own, torch.zeros((), dtype=torch.bool, device="cuda")))
    torch.cuda.synchronize()
    start, bad = threading.Barrier(2), []

    def work(c, q, o, lse, ws, desc, pdesc, own, off):
        stream = torch.cuda.Stream()
        try:
            with torch.cuda.stream(stream):
                o2, l2 = torch.zeros_like(o), torch.zeros_like(lse)
                start.wait(60)
                for _ in range(200):
                    o2.zero_()
                    l2.zero_()
                    G.gsa_paged_attend(desc, pdesc, 1, q, *c.args(), None, own, o2, l2, ws)
                    off |= (o2 != o).any() | (l2 != lse).any()
                stream.synchronize()
        except Exception as e:  # reported by the test's own thread
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
    assert not any(bool(j[-1]) for j in jobs)


@pytest.mark.parametrize("levels", [1, 2])
@pytest.mark.parametrize("exclude", [False, True])
def test_hierarchical_selections_feed_the_paged_unfold(levels, exclude):
    """hgsa_select / hgsa2_select, then gsa_paged_unfold: the outputs of gsa_unfold_attend on the same selection and
    partial, over raw rows that hold the codes' values exactly (e4m3 codes, power-of-two scales, bf16)."""
    B, hq, hkv, d, chunk, N = 2, 8, 2, 64, 8, 64
    c = Cache([N * chunk + 5, N * chunk + 1], hkv, d, chunk, 32, "e4m3", seed=3)
    g = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, gk, gv, mk, mv, m2k, m2v = rnd(B, hq, d), *(rnd(B, hkv, n, d) for n in (N, N, 16, 16, 4, 4))
    n = torch.full((B,), N, dtype=torch.int32, device="cuda")
    own = torch.tensor([5, 1], dtype=torch.int32, device="cuda")
    desc = G.make_desc(B, hq, hkv, d, chunk, N, c.cap, 6, exclude)
    pdesc = G.make_pdesc(G.GSA_E4M3, c.page, c.n_pages, c.max_pages)
    raw = {kv: torch.zeros((B, hkv, c.cap, d), dtype=torch.bfloat16, device="cuda") for kv in "kv"}
    for kv in "kv":
        for b in range(B):
            raw[kv][b, :, :c.lens[b]] = c.rows(kv, b, c.lens[b]).to(torch.bfloat16)
            assert torch.equal(raw[kv][b, :, :c.lens[b]].double(), c.rows(kv, b, c.lens[b]))
    h1 = G.make_hdesc(4, 3, 16)
    hd = h1 if levels == 1 else G.make_h2desc(h1, G.make_hdesc(4, 2, 4))
    ws = torch.empty(G.gsa_workspace_bytes(desc, (G.GSA_OP_HGSA, G.GSA_OP_HGSA2)[levels - 1], hd), dtype=torch.uint8,
                     device="cuda")
    G.gsa_workspace_init(ws)
    idx = lambda k: torch.empty((B, hq, k), dtype=torch.int32, device="cuda")  # noqa: E731
    si, ss = idx(6), torch.empty((B, hq, 6), device="cuda")
    outs = []
    for paged in (True, False):
        if levels == 1:
            G.hgsa_select(desc, hd, q, mk, mv, gk, gv, n, idx(3), si, ss, ws)
        else:
            G.hgsa2_select(desc, hd, q, m2k, m2v, mk, mv, gk, gv, n, idx(2), idx(3), si, ss, ws)
        prior = G.GSA_PRIOR_NONE if exclude else (G.GSA_PRIOR_HGSA, G.GSA_PRIOR_HGSA2)[levels - 1]
        o, lse = torch.empty((B, hq, d), device="cuda"), torch.empty((B, hq), device="cuda")
        if paged:
            G.gsa_paged_unfold(desc, pdesc, q, *c.args(), gv, n, own, si, ss, prior, o, lse, ws)
        else:
            G.gsa_unfold_attend(desc, q, raw["k"], raw["v"], gv, n, own, si, ss, prior, o, lse, ws)
        outs.append((o, lse))
    # The partial and the selection are the same bits.  Both unfolds' logits sum bf16 products in fp32 (reach below
    # 2^6 here: 2^-15 of a weight), the unpaged one's weights are two bf16 terms (2^-16): 2^-13 of the largest value
    # covers twice their sum.
    vmax = max(float(raw["v"].abs().max()), float(gv.abs().max()), float(mv.abs().max()))
    assert float((outs[0][0] - outs[1][0]).abs().max()) <= 2.0 ** -13 * vmax
    assert float((outs[0][1] - outs[1][1]).abs().max()) <= 2.0 ** -14
    assert G.gsa_workspace_status(ws) == 0
