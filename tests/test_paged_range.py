"""The paged readers at the ends of their range: scales of V far apart inside and across tiles, weights whose values
cancel, queries with elements of very different sizes.  Bounds are relative to each output's own sum of |weight x value|,
dim by dim, so that a large value elsewhere hides nothing."""
import math

import pytest
import torch

from _paged import Cache
from test_paged_attend import DT, descs, run_attend

pytestmark = pytest.mark.gpu

G = None
LOG2E = math.log2(math.e)


@pytest.fixture(scope="module", autouse=True)
def _setup():
    global G
    from long_context_gsa_b200 import build
    build.build_library()
    import long_context_gsa_b200 as G_
    import test_paged_attend as A
    G = A.G = G_


def strict(got, got_lse, q, k, v, scale, what, *, bf16=False, extra=None):
    """One row against 64 bits: off by rel * sum p |v| in each dim.

    A base-2 logit is off by dz: products of the operands' parts are exact, their fp32 sums over d / 16 products may
    truncate at 2^-22 of the largest partial sum each, three scalings round at 2^-24.  The query's last part ends at
    2^-28 of its largest element (int8 keys; further down for e4m3).  A weight is off by ln 2 dz relative to itself,
    so is the sum of them; the exponential and the fp32 sums add 2^-19.  Weights enter the products with an error of
    2^-24 of themselves, or 2^-25 of the largest weight among keys whose scales lie within 2^10 of theirs."""
    d = q.shape[-1]
    z = (k @ q) * scale
    dz = 0.0
    if len(k):
        dz = (d / 16 + 3) * 2.0 ** -22 * float((k.abs() @ q.abs()).max()) * scale * LOG2E
        dz += 2.0 ** -28 * float(q.abs().max() * k.abs().sum(-1).max()) * scale * LOG2E
    if extra is not None:
        z, v = torch.cat([z, extra[0]]), torch.cat([v, extra[1]])
    lse = torch.logsumexp(z, 0)
    p = torch.exp(z - lse)[:, None]
    ref, size = (p * v).sum(0), (p * v.abs()).sum(0)
    lim = (1.4 * dz + 2.0 ** -19) * size
    if len(k):  # keys whose scales may share a reference (a row may lack its block's largest: 2^9)
        pk, s = p[:len(k), 0], v[:len(k)].abs().amax(-1)
        near = (s[None] < s[:, None] * 2.0 ** 19) & (s[None] * 2.0 ** 19 > s[:, None])
        lim = lim + 2.0 ** -25 * ((near * pk[None]).amax(1)[:, None] * v[:len(k)].abs()).sum(0)
    if bf16:
        lim = lim + 2.0 ** -8 * (ref.abs() + lim)
    err = (got.double() - ref).abs()
    worst = float((err - lim).max())
    assert worst <= 0, f"{what}: {worst:.3e} over the bound, error {float(err.max()):.3e}"
    assert abs(float(got_lse) - float(lse)) <= dz + 2.0 ** -19 + 2.0 ** -21 * abs(float(lse)), f"{what}: lse"
    return ref


def check(c, hq, n_q, q, o, lse, out, scale=0.0):
    s = scale or 1 / math.sqrt(c.d)
    for b, n in enumerate(c.lens):
        k, v = c.rows("k", b, n), c.rows("v", b, n)
        for i in range(n_q):
            end = n - (n_q - 1) + i
            for h in range(hq):
                kv = h // (hq // c.hkv)
                strict(o[b, i, h], lse[b, i, h], q[b, i, h].double(), k[kv, :end], v[kv, :end], s,
                       f"seq {b} query {i} head {h}", bf16=out == "bf16")


def set_block(c, kv, b, blk, f):
    """The scale of block blk of sequence b times f (every head)."""
    per = c.page // c.chunk
    c.scales[kv][int(c.table[b, blk // per]), :, blk % per] *= f


def call(c, hq, q, *, dtype, out):
    desc, pdesc, ws = descs(c, hq, dtype=dtype, out=out)
    B, n_q = len(c.lens), q.shape[1]
    o = torch.full((B, n_q, hq, c.d), float("nan"), dtype=DT[out], device="cuda")
    lse = torch.full((B, n_q, hq), float("nan"), device="cuda")
    own = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    G.gsa_paged_attend(desc, pdesc, n_q, q, *c.args(), None, own, o, lse, ws)
    assert G.gsa_workspace_status(ws) == 0
    return o, lse


@pytest.mark.parametrize("fmt,d,out", [("e4m3", 64, "f32"), ("i8", 128, "f32"), ("i8", 64, "bf16"), ("e4m3", 128, "bf16")])
@pytest.mark.parametrize("apart", [10, 11, 20, 40, 90])
def test_scales_far_apart_in_a_tile(fmt, d, out, apart):
    """Neighbouring blocks of 8 rows whose values differ by 2^apart; the keys make the small ones weigh as much, e^-30
    or e^-60 times as much, or more (a head each)."""
    c = Cache([24, 96, 700], 1, d, 8, 64, fmt, seed=apart)
    for b, n in enumerate(c.lens):
        for blk in range(-(-n // 8)):
            set_block(c, "v", b, blk, 2.0 ** (-apart * (blk % 3) / 2 + apart / 2))
    ones = torch.ones((c.n_pages, 1, c.page, d), device="cuda")
    c.pages["k"] = ones.to(c.pages["k"].dtype)
    for b, n in enumerate(c.lens):
        per = c.page // 8
        for blk in range(-(-n // 8)):  # logits 0, 30 and 60 at a query of ones
            c.scales["k"][int(c.table[b, blk // per]), :, blk % per] = 30.0 * (blk % 3) / math.sqrt(d)
    q = torch.tensor([1.0, 0.0, -1.0, 0.25], device="cuda")[None, None, :, None].expand(3, 1, 4, d)
    q = q.to(torch.bfloat16).contiguous()
    o, lse = call(c, 4, q, dtype="bf16", out=out)
    check(c, 4, 1, q, o, lse, out)


@pytest.mark.parametrize("fmt,d,dtype,n_q", [("e4m3", 64, "bf16", 1), ("i8", 128, "f32", 1), ("i8", 64, "bf16", 5),
                                            ("e4m3", 128, "f32", 5)])
def test_scales_of_any_size(fmt, d, dtype, n_q):
    """Random scales over a hundred octaves, within a tile and from tile to tile."""
    c = Cache([300, 47, 2100], 2, d, 8, 24, fmt, seed=d + n_q)
    g = torch.Generator(device="cuda").manual_seed(3)
    c.scales["v"] *= torch.exp2(100 * torch.rand(c.scales["v"].shape, generator=g, device="cuda") - 50).round_()
    c.scales["v"][torch.rand(c.scales["v"].shape, generator=g, device="cuda") < 0.1] = 0.0  # and blocks of zeros
    q, o, lse, ws, _ = run_attend(c, 8, n_q, dtype=dtype)
    check(c, 8, n_q, q, o, lse, "f32")
    assert G.gsa_workspace_status(ws) == 0


def test_a_later_tokens_values_do_not_touch_earlier_queries():
    """Of 6 drafted tokens the last has values 2^60 times as large: the queries that do not see it keep their bits."""
    outs = []
    for f in (1.0, 2.0 ** 60):
        c = Cache([41], 1, 64, 8, 8, "e4m3", seed=4)
        set_block(c, "v", 0, 5, f)  # row 40
        q, o, lse, _, _ = run_attend(c, 8, 6)
        check(c, 8, 6, q, o, lse, "f32")
        outs.append(o)
    assert float((outs[0][0, :5] - outs[1][0, :5]).abs().max()) <= 2.0 ** -20 * float(outs[0][0, :5].abs().max())


@pytest.mark.parametrize("exclude", [True, False])
@pytest.mark.parametrize("fmt,d,chunk", [("e4m3", 64, 8), ("i8", 128, 16)])
def test_unfold_of_chunks_with_scales_far_apart(fmt, d, chunk, exclude):
    """Selected chunks that share tiles and splits, values 2^40 apart; alone and in the fused step."""
    B, hq, hkv, topk, N = 2, 4, 2, 20, 60
    c = Cache([chunk * N + 3, chunk * N + chunk - 1], hkv, d, chunk, 2 * chunk, fmt, seed=chunk)
    for b in range(B):
        for blk in range(N + 1):
            set_block(c, "v", b, blk, 2.0 ** (40 * (blk % 3 - 1)))
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    desc, pdesc, ws = descs(c, hq, topk=topk, n_max=N, exclude=exclude)
    q, gk, gv = rnd(B, hq, d), rnd(B, hkv, N, d), rnd(B, hkv, N, d)
    n = torch.full((B,), N, dtype=torch.int32, device="cuda")
    own = torch.tensor([3, chunk - 1], dtype=torch.int32, device="cuda")
    o, lse = torch.empty((B, hq, d), device="cuda"), torch.empty((B, hq), device="cuda")
    sel = torch.empty((B, hq, topk), dtype=torch.int32, device="cuda")
    score = torch.empty((B, hq, topk), device="cuda")
    G.gsa_paged_decode(desc, pdesc, q, gk, gv, *c.args(), n, own, o, lse, sel, score, ws)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    if not exclude:
        G.gsa_score_gists(desc, q, gk, gv, n, torch.empty((B, hq, N), device="cuda"), ws)
    G.gsa_paged_unfold(desc, pdesc, q, *c.args(), gv, n, own, sel, score,
                       G.GSA_PRIOR_NONE if exclude else G.GSA_PRIOR_GISTS, o2, lse2, ws)
    assert G.gsa_workspace_status(ws) == 0
    s = 1 / math.sqrt(d)
    for b in range(B):
        rows = c.lens[b]
        k, v = c.rows("k", b, rows), c.rows("v", b, rows)
        for h in range(hq):
            kv, qd, ids = h // (hq // hkv), q[b, h].double(), sel[b, h].long()
            at = torch.cat([(ids[:, None] * chunk + torch.arange(chunk, device="cuda")).flatten(),
                            torch.arange(N * chunk, rows, device="cuda")])
            pick = ids if exclude else torch.arange(N, device="cuda")
            gz = score[b, h].double() if exclude else gk[b, kv].double() @ qd * s
            for got, ln in ((o, lse), (o2, lse2)):
                # the gists' values are 2^-40 of the largest rows', their weights two bf16 terms (2^-16) beside a prior
                want = strict_parts(qd, k[kv, at], v[kv, at], gz, gv[b, kv, pick].double(), s)
                err = (got[b, h].double() - want[0]).abs()
                assert bool((err <= want[1]).all()), f"{b} {h}: {float((err - want[1]).max()):.3e} over the bound"


def strict_parts(q, k, v, gz, gv, s):
    """Output and bound of rows and gists together, as in strict (2^-14 relative covers the logits here: their reach
    is below 2^5, (8 + 3) 2^-22 2^5 1.4 < 2^-13.0; the gists' 2^-16 comes on top)."""
    z = torch.cat([(k @ q) * s, gz])
    x = torch.cat([v, gv])
    p = torch.exp(z - torch.logsumexp(z, 0))[:, None]
    return (p * x).sum(0), (2.0 ** -12.5) * (p * x.abs()).sum(0)


@pytest.mark.parametrize("fmt,d", [("e4m3", 64), ("i8", 64), ("e4m3", 128), ("i8", 128)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_values_that_cancel(fmt, d, out):
    """Rows in pairs of opposite values under near-equal weights: the output is small beside its terms, so the weights'
    rounding shows whatever the output's type."""
    c = Cache([34, 130, 600], 1, d, 2, 32, fmt, seed=8, std=0.5)
    codes = c.pages["v"].double()
    codes[:, :, 1::2] = -codes[:, :, ::2]
    c.pages["v"] = codes.to(c.pages["v"].dtype)
    g = torch.Generator(device="cuda").manual_seed(9)
    q = (torch.randn((3, 1, 8, d), generator=g, device="cuda") * 0.5).to(torch.bfloat16)
    o, lse = call(c, 8, q, dtype="bf16", out=out)
    check(c, 8, 1, q, o, lse, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_query_with_one_large_element(fmt, dtype):
    """An element 2^8 times the others where the keys are 0: the others still count to their last bits."""
    c = Cache([40, 333], 1, 64, 8, 32, fmt, seed=10)
    codes = c.pages["k"].double()
    codes[..., 5] = 0
    c.pages["k"] = codes.to(c.pages["k"].dtype)
    g = torch.Generator(device="cuda").manual_seed(11)
    q = torch.randn((2, 1, 4, 64), generator=g, device="cuda")
    q[..., 5] = 700.0
    q = q.to(DT[dtype])
    o, lse = call(c, 4, q, dtype=dtype, out="f32")
    check(c, 4, 1, q, o, lse, "f32")


def test_logits_whose_factors_pass_fp32():
    """Keys of 0 in a block with a scale of 2^120 under queries of 2^40: logits of 0, though the product of the two
    factors is beyond fp32."""
    for fmt in ("i8", "e4m3"):
        c = Cache([24], 1, 64, 8, 8, fmt, seed=12)
        c.pages["k"] = torch.zeros((c.n_pages, 1, 8, 64), device="cuda").to(c.pages["k"].dtype)
        c.scales["k"].fill_(2.0 ** 120)
        q = torch.full((1, 1, 2, 64), 2.0 ** 40, device="cuda", dtype=torch.bfloat16)
        o, lse = call(c, 2, q, dtype="bf16", out="f32")
        v = c.rows("v", 0, 24)[0]
        assert bool(((o[0, 0].double() - v.mean(0)).abs() <= 2.0 ** -19 * v.abs().mean(0)).all())
        assert bool(((lse - math.log(24)).abs() <= 2.0 ** -19).all())


@pytest.mark.parametrize("fmt,d,n_q", [("e4m3", 64, 1), ("i8", 128, 1), ("i8", 64, 4), ("e4m3", 128, 4)])
def test_many_segments_each_cut(fmt, d, n_q):
    """16 sequences x 4 kv heads, most of them shared by a few CTAs: few records to a segment."""
    c = Cache([2600 + 37 * i for i in range(14)] + [0, 90], 4, d, 16, 48, fmt, seed=n_q)
    q, o, lse, ws, _ = run_attend(c, 16, n_q, dtype="bf16")
    assert not o[14].any() and bool((lse[14] == -math.inf).all())
    for b in (0, 3, 6, 9, 13, 15):
        k, v = c.rows("k", b, c.lens[b]), c.rows("v", b, c.lens[b])
        for i in range(n_q):
            end = c.lens[b] - (n_q - 1) + i
            for h in range(0, 16, 3):
                strict(o[b, i, h], lse[b, i, h], q[b, i, h].double(), k[h // 4, :end], v[h // 4, :end],
                       1 / math.sqrt(d), f"seq {b} query {i} head {h}")
    assert G.gsa_workspace_status(ws) == 0


def test_nothing_cached_anywhere():
    """A batch without a single row: zeros and empty sums, in one call and in a batch of the largest size."""
    for lens in ([0], [0] * 8192):
        c = Cache.__new__(Cache)
        c.lens, c.hkv, c.d, c.chunk, c.page, c.fmt, c.cap = lens, 1, 64, 8, 8, "i8", 8
        c.max_pages, c.n_pages = 1, 1
        c.table = torch.full((len(lens), 1), -1, dtype=torch.int32, device="cuda")
        c.pages = {kv: torch.full((1, 1, 8, 64), -128, dtype=torch.int8, device="cuda") for kv in "kv"}
        c.scales = {kv: torch.full((1, 1, 1), float("nan"), device="cuda") for kv in "kv"}
        q, o, lse, ws, _ = run_attend(c, 2, 2)
        assert not o.any() and bool((lse == -math.inf).all()) and G.gsa_workspace_status(ws) == 0
