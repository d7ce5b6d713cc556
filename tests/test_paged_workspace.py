"""One workspace under several descriptors: what a paged call leaves in it, or finds there, does not reach the next."""
import pytest
import torch

from _paged import Cache
from test_paged_append import Pool, append, check_append
from test_paged_attend import check_unfold, code_of, descs, run_unfold

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
