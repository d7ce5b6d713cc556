"""gsa_paged_append (rotation, 8-bit blocks, pages) against 64-bit formulas,
and the paged calls run together as a serving loop runs them."""
import math

import pytest
import torch

from _paged import CODE, Cache, block_scale
from test_paged_attend import check_row, code_of

pytestmark = pytest.mark.gpu

G = None
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    global G
    from long_context_gsa_b200 import build
    build.build_library()
    import long_context_gsa_b200 as G_
    import test_paged_attend as A
    G = A.G = G_


def rotate(x, pos, inv_freq, inter):
    """[T, heads, d] in 64 bits, the first 2 * len(inv_freq) dims turned as complex numbers."""
    y = x.double().clone()
    rot = 2 * len(inv_freq)
    if rot:
        ang = pos.double()[:, None] * inv_freq.double()
        turn = torch.polar(torch.ones_like(ang), ang)[:, None, :]
        ia = torch.arange(0, rot, 2, device=x.device) if inter else torch.arange(rot // 2, device=x.device)
        ib = ia + (1 if inter else rot // 2)
        w = torch.complex(y[..., ia], y[..., ib]) * turn
        y[..., ia], y[..., ib] = w.real, w.imag
    return y


def turn_slack(x, rot, inter):
    """Error of a turned value: cosine and sine within 2^-22 and two roundings of products, each at most 2^-21 of
    |x| + |y| of the pair together (0 for dims that are not turned)."""
    a = x.double().abs()
    s = torch.zeros_like(a)
    if rot:
        if inter:
            both = a[..., 0:rot:2] + a[..., 1:rot:2]
            s[..., 0:rot:2] = s[..., 1:rot:2] = both
        else:
            both = a[..., :rot // 2] + a[..., rot // 2:rot]
            s[..., :rot // 2] = s[..., rot // 2:rot] = both
    return s * 2.0 ** -21


class Pool:
    """An empty pool filled with garbage, and what should be in it (64 bits)."""

    def __init__(self, B, hkv, d, chunk, page, cap, fmt, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.hkv, self.d, self.chunk, self.page, self.cap, self.fmt = B, hkv, d, chunk, page, cap, fmt
        self.max_pages = -(-cap // page)
        self.n_pages = B * self.max_pages + 2
        self.table = torch.randperm(self.n_pages, generator=g)[:B * self.max_pages].view(B, -1).to(torch.int32).cuda()
        self.pages = {kv: torch.full((self.n_pages, hkv, page, d), 99 if fmt != "e4m3" else 7.0).to(CODE[fmt]).cuda()
                      for kv in "kv"}
        coded = fmt in ("i8", "e4m3")
        self.scales = {kv: torch.full((self.n_pages, hkv, page // chunk), 5.0, device="cuda") if coded else None
                       for kv in "kv"}

    def args(self):
        return self.table, self.pages["k"], self.pages["v"], self.scales["k"], self.scales["v"]

    rows = Cache.rows

    def row_scale(self, kv, b, n):
        """[hkv, n] scales of the first n rows."""
        s = torch.cat([self.scales[kv][int(self.table[b, p])].repeat_interleave(self.chunk, -1)
                       for p in range(-(-n // self.page))], -1)
        return s[:, :n].double()

    def desc(self, hq, dtype, **kw):
        desc = G.make_desc(self.B, hq, self.hkv, self.d, self.chunk, kw.get("n_max", 1), self.cap, kw.get("topk", 0),
                           kw.get("exclude", True), 0.0, code_of(dtype), kw.get("out", G.GSA_F32))
        pdesc = G.make_pdesc(code_of(self.fmt), self.page, self.n_pages, self.max_pages)
        ws = torch.empty(G.gsa_workspace_bytes(desc, G.GSA_OP_PAGED), dtype=torch.uint8, device="cuda")
        G.gsa_workspace_init(ws)
        return desc, pdesc, ws


def check_rows(got, want, slack, scale, fmt, rounds, what):
    """Stored values against 64-bit ones.  One rounding is half a step: int8 s / 2; e4m3 2^-4 of the value, at least
    half the subnormal step s 2^-10; bf16 2^-8, fp32 2^-24 of the value.  `rounds`: how often a row can have been
    rounded (rows of a part-filled block whose scale grew).  The quotient x / s of int8 is a product with a rounded
    reciprocal: 2^-22 of the value more."""
    if fmt == "i8":
        one = 0.5 * scale
    elif fmt == "e4m3":
        one = torch.maximum(want.abs() * 2.0 ** -4, scale * 2.0 ** -10)
    else:
        one = want.abs() * (2.0 ** -8 if fmt == "bf16" else 2.0 ** -24)
    lim = rounds * one * (1 + 2.0 ** -4) + slack + want.abs() * 2.0 ** -22
    err = (got - want).abs()
    assert bool((err <= lim).all()), f"{what}: {float((err - lim).max()):.3e} over the bound"


def append(p, hq, lens, new, *, dtype="bf16", rot=0, inter=False, advance=False, pos=None, seed=0, strided=False,
           uniform=False, n_gists=None, std=1.0, state=None, pad=0, with_q=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, d, hkv = sum(new), p.d, p.hkv
    width = (hq + 2 * hkv) * d
    fused = (torch.randn((T + pad, width), generator=g, device="cuda") * std).to(DT[dtype])
    parts = fused.split([hq * d, hkv * d, hkv * d], 1)
    q, k, v = [(x if strided else x.contiguous()).view(T + pad, x.shape[1] // d, d) for x in parts]
    desc, pdesc, ws = state or p.desc(hq, dtype)
    st = width if strided else 0
    adesc = G.make_append_desc(T + pad, rot, inter, advance, st, st, st)
    inv = torch.tensor([10000.0 ** (-2 * i / max(rot, 1)) for i in range(rot // 2)], dtype=torch.float32, device="cuda")
    cu = None if uniform else torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device="cuda")
    own = torch.tensor(lens, dtype=torch.int32, device="cuda") if not torch.is_tensor(lens) else lens
    q_out = torch.full((T + pad, hq, d), 77.0, dtype=DT[dtype], device="cuda")
    G.gsa_paged_append(desc, pdesc, adesc, q if with_q else None, k, v, cu, pos, inv if rot else None, p.table, n_gists,
                       own, *p.args()[1:], q_out if with_q else None, ws)
    return dict(q=q, k=k, v=v, inv=inv, q_out=q_out, own=own, ws=ws, rot=rot, inter=inter)


def check_append(p, r, lens, new, pos=None, rounds=None, drop=lambda b, row: False):
    at, dt = 0, r["k"].dtype
    for b, (n, t) in enumerate(zip(lens, new)):
        sl = slice(at, at + t)
        at += t
        if t == 0:
            continue
        ps = pos[sl] if pos is not None else torch.arange(n, n + t, device="cuda")
        turned = rotate(r["q"][sl], ps, r["inv"], r["inter"])
        qs = turn_slack(r["q"][sl], r["rot"], r["inter"])
        lim = turned.abs() * (2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24) * (1 + 2.0 ** -8) + qs
        assert bool(((r["q_out"][sl].double() - turned).abs() <= lim).all()), f"q of seq {b}"
        keep = torch.tensor([n + i < p.cap and not drop(b, n + i) for i in range(t)], device="cuda")
        for kv, x in (("k", rotate(r["k"][sl], ps, r["inv"], r["inter"])), ("v", r["v"][sl].double())):
            slack = turn_slack(r["k"][sl], r["rot"], r["inter"]) if kv == "k" else torch.zeros_like(x)
            end = min(n + t, p.cap)
            keep_ = keep[:end - n]
            got, sc = p.rows(kv, b, end)[:, n:].transpose(0, 1)[keep_], None
            if p.scales[kv] is not None:
                sc = p.row_scale(kv, b, end)[:, n:].transpose(0, 1)[keep_][..., None]
            check_rows(got, x[:end - n][keep_], slack[:end - n][keep_], sc, p.fmt, rounds or 1, f"{kv} of seq {b}")
            if sc is None or rounds:
                continue
            # scales of blocks that this call began (with `rounds`, later calls may have raised them)
            for blk in range(-(-n // p.chunk), -(-end // p.chunk)):
                lo, hi = max(blk * p.chunk, n) - n, min((blk + 1) * p.chunk, end) - n
                if any(drop(b, n + i) for i in range(lo, hi)):
                    continue
                want = block_scale(x[lo:hi].abs().amax((0, 2)), p.fmt)
                have = p.row_scale(kv, b, end)[:, n + lo]
                # int8: the turned maximum's error and the division; e4m3: the same power of two (random maxima are
                # nowhere near 448 2^n)
                lim = want * (2.0 ** -20 if p.fmt == "i8" else 0)
                assert bool(((have - want).abs() <= lim).all()), f"scale {kv} {b} {blk}"


APPEND = [
    # fmt, dtype, hq, hkv, d, chunk, page, lens, new, rot, inter, strided
    ("e4m3", "bf16", 8, 2, 64, 8, 64, [0, 3, 7, 8, 61], [1, 1, 1, 1, 1], 64, False, False),
    ("i8", "bf16", 7, 1, 128, 16, 16, [0, 15, 33], [40, 1, 90], 128, False, True),
    ("e4m3", "bf16", 4, 4, 128, 24, 72, [5, 0, 23, 100], [77, 0, 2, 24], 32, True, True),
    ("i8", "f32", 2, 1, 64, 7, 21, [0, 6, 13], [50, 1, 8], 16, False, False),
    ("e4m3", "f32", 1, 1, 128, 64, 64, [1, 70], [300, 129], 112, True, False),
    ("i8", "bf16", 3, 3, 64, 1, 2, [0, 5], [9, 1], 0, False, False),
    ("bf16", "bf16", 4, 2, 64, 8, 32, [3, 0], [30, 8], 64, False, True),
    ("f32", "f32", 4, 2, 128, 16, 16, [17, 0, 1], [1, 65, 0], 48, True, False),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{c[0]}_{c[1]}_d{c[4]}_c{c[5]}_p{c[6]}_rot{c[9]}")
def test_append_from_what_is_held(case):
    """Rows behind what each sequence holds (itself appended first), ragged, in every layout."""
    fmt, dtype, hq, hkv, d, chunk, page, lens, new, rot, inter, strided = case
    p = Pool(len(lens), hkv, d, chunk, page, max(a + b for a, b in zip(lens, new)) + 3, fmt, seed=d + chunk)
    r0 = append(p, hq, [0] * len(lens), lens, dtype=dtype, rot=rot, inter=inter, seed=1)
    check_append(p, r0, [0] * len(lens), lens)
    before = {kv: p.pages[kv].view(torch.uint8).clone() for kv in "kv"}
    r = append(p, hq, lens, new, dtype=dtype, rot=rot, inter=inter, seed=2, strided=strided)
    check_append(p, r, lens, new)
    check_append(p, r0, [0] * len(lens), lens, rounds=2)  # a part-filled block may have been rounded again
    # nothing else changed: rows past the end, other blocks, other pages
    touched = torch.zeros((p.n_pages, page), dtype=torch.bool, device="cuda")
    for b, (n, t) in enumerate(zip(lens, new)):
        if t:
            for row in range(n - n % chunk, n + t):
                touched[int(p.table[b, row // page]), row % page] = True
    for kv in "kv":
        same = (p.pages[kv].view(torch.uint8) == before[kv]).all(-1).all(1)
        assert bool((same | touched).all())
    assert G.gsa_workspace_status(r["ws"]) == 0 and r["own"].tolist() == lens


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_token_by_token_and_advance(fmt):
    """A decode loop's single tokens: lengths advance on the device, blocks are rounded at most once per growth."""
    p = Pool(3, 2, 64, 8, 16, 64, fmt)
    state = p.desc(4, "bf16")
    own = torch.tensor([0, 5, 11], dtype=torch.int32, device="cuda")
    r0 = append(p, 4, [0, 0, 0], [0, 5, 11], rot=64, seed=3, state=state)
    steps = []
    for i in range(20):
        # tokens grow, so the scales of part-filled blocks do too
        steps.append(append(p, 4, own, [1, 1, 1], rot=64, seed=10 + i, advance=True, uniform=True, state=state,
                            std=1.0 + 0.3 * i))
    assert own.tolist() == [20, 25, 31]
    for i, r in enumerate(steps):
        check_append_one(p, r, [i, 5 + i, 11 + i])
    check_append(p, r0, [0, 0, 0], [0, 5, 11], rounds=8)
    assert G.gsa_workspace_status(state[2]) == 0


def check_append_one(p, r, lens):
    """Single tokens whose blocks may have been rounded again up to chunk - 1 times since."""
    for b, n in enumerate(lens):
        ps = torch.tensor([n], device="cuda")
        for kv, x in (("k", rotate(r["k"][b:b + 1], ps, r["inv"], r["inter"])), ("v", r["v"][b:b + 1].double())):
            got = p.rows(kv, b, n + 1)[:, n:].transpose(0, 1)
            sc = p.row_scale(kv, b, n + 1)[:, n:].transpose(0, 1)[..., None]
            slack = turn_slack(r["k"][b:b + 1], r["rot"], r["inter"])
            # int8: half a final step at most for each growth.  e4m3's power-of-two steps lose only in the subnormals:
            # one rounding of the value, then half steps that double up to the final one, 2 of it together
            check_rows(got, x, slack, sc, p.fmt, p.chunk if p.fmt == "i8" else 3, f"{kv} seq {b} row {n}")


def test_far_positions():
    """Positions of a very long context, given explicitly: fp32 angles would be off by radians."""
    p = Pool(2, 1, 64, 8, 64, 40, "f32")
    pos = torch.tensor([(1 << 30) + 7 * i for i in range(20)] + [2000003 + i for i in range(13)], dtype=torch.int32,
                       device="cuda")
    r = append(p, 2, [0, 0], [20, 13], dtype="f32", rot=64, pos=pos)
    check_append(p, r, [0, 0], [20, 13], pos=pos)


def test_rows_past_the_capacity_and_bad_pages():
    p = Pool(2, 2, 64, 8, 16, 40, "e4m3")
    r = append(p, 4, [30, 8], [20, 16], rot=64, advance=True)
    assert G.gsa_workspace_status(r["ws"]) == G.GSA_DEVERR_CAPACITY
    assert r["own"].tolist() == [40, 24]
    assert bool((r["q_out"][10:20] == 77).all())  # dropped tokens' queries are not written
    p = Pool(2, 2, 64, 8, 16, 40, "e4m3")
    p.table[1, 1] = p.n_pages + 4
    r = append(p, 4, [0, 0], [20, 40], rot=64)
    assert G.gsa_workspace_status(r["ws"]) == G.GSA_DEVERR_BAD_INDEX
    p.table[1, 1] = p.table[1, 0]  # any page: its rows are left out below
    check_append(p, r, [0, 0], [20, 40], drop=lambda b, row: b == 1 and 16 <= row < 32)


def test_padded_rows_and_empty_calls_leave_everything():
    p = Pool(2, 1, 64, 8, 16, 64, "i8")
    r = append(p, 2, [0, 9], [5, 4], rot=16, pad=30)
    check_append(p, r, [0, 9], [5, 4], rounds=2)
    assert bool((r["q_out"][9:] == 77).all())
    before = [p.pages[kv].clone() for kv in "kv"] + [p.scales[kv].clone() for kv in "kv"]
    r = append(p, 2, [5, 13], [0, 0], rot=16, pad=3, advance=True)
    assert r["own"].tolist() == [5, 13]
    append(p, 2, [5, 13], [0, 0], rot=16)
    for a, b in zip(before, [p.pages[kv] for kv in "kv"] + [p.scales[kv] for kv in "kv"]):
        assert torch.equal(a, b)


def test_zero_tiny_huge_and_nonfinite_blocks():
    for fmt in ("i8", "e4m3"):
        p = Pool(1, 1, 64, 8, 8, 64, fmt)
        state = p.desc(1, "f32")
        desc, pdesc, ws = state
        g = torch.Generator(device="cuda").manual_seed(4)
        k = torch.randn((40, 1, 64), generator=g, device="cuda")
        k[0:8] = 0
        k[8:16] *= 1e-32          # below 2^-100: kept as zeros
        k[16:24] *= 1e-27
        k[24:32] *= 1e37
        k[35, 0, 3] = math.inf
        v = k.clone()
        v[35, 0, 3] = math.nan
        own = torch.zeros(1, dtype=torch.int32, device="cuda")
        G.gsa_paged_append(desc, pdesc, G.make_append_desc(40), None, k, v, None, None, None, p.table, None, own,
                           *p.args()[1:], None, ws)
        for kv, x in (("k", k), ("v", v)):
            got, s = p.rows(kv, 0, 40)[0], p.row_scale(kv, 0, 40)[0]
            assert bool((s[:16] == 0).all()) and bool((got[:16] == 0).all())
            assert bool(torch.isnan(got[32:40]).all()) and bool(torch.isnan(s[32:40]).all())
            check_rows(got[16:32], x[16:32, 0].double(), 0.0, s[16:32, None], fmt, 1, f"{fmt} {kv}")
        # a NaN block stays one when rows join; the first row of a block starts it anew
        own.fill_(35)
        G.gsa_paged_append(desc, pdesc, G.make_append_desc(1), None, k[:1] + 1, v[:1] + 1, None, None, None, p.table,
                           None, own, *p.args()[1:], None, ws)
        assert bool(torch.isnan(p.row_scale("k", 0, 40)[0, 32:]).all())
        own.fill_(32)
        G.gsa_paged_append(desc, pdesc, G.make_append_desc(8), None, k[:8] + 1, v[:8] + 1, None, None, None, p.table,
                           None, own, *p.args()[1:], None, ws)
        check_rows(p.rows("k", 0, 40)[0, 32:], torch.ones((8, 64), dtype=torch.float64, device="cuda"), 0.0,
                   p.row_scale("k", 0, 40)[0, 32:, None], fmt, 1, "block begun anew")


def test_append_without_queries_many_sequences():
    """600 sequences (prefix sums over several passes), no queries, uniform counts."""
    B = 600
    p = Pool(B, 1, 64, 8, 8, 24, "e4m3")
    lens = [i % 13 for i in range(B)]
    append(p, 1, [0] * B, lens, rot=64, seed=1)
    r = append(p, 1, lens, [3] * B, rot=64, seed=2, uniform=True, with_q=False)
    pos = torch.tensor([n + i for n in lens for i in range(3)], device="cuda")
    r["q_out"] = rotate(r["q"], pos, r["inv"], False).to(r["k"].dtype)  # not written by this call
    check_append(p, r, lens, [3] * B)


def test_unpaged_cache_is_a_pool_of_one_page_a_sequence():
    """page = t_max, page_table[b] = b: the raw_k / raw_v arrays of gsa_decode, with rows counted from n_gists."""
    B, hkv, d, chunk, t_max = 2, 2, 64, 8, 64
    raw_k, raw_v = (torch.zeros((B, hkv, t_max, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    p = Pool(B, hkv, d, chunk, t_max, t_max, "bf16")
    p.n_pages, p.max_pages = B, 1
    p.table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    p.pages = {"k": raw_k, "v": raw_v}
    n = torch.tensor([3, 5], dtype=torch.int32, device="cuda")
    r = append(p, 4, [2, 7], [4, 9], rot=64, n_gists=n, state=p.desc(4, "bf16", n_max=7))
    check_append(p, r, [3 * 8 + 2, 5 * 8 + 7], [4, 9])


# ------------------------------------------------------------- together
@pytest.mark.parametrize("fmt,dtype,d,hq,hkv,chunk,page", [
    ("e4m3", "bf16", 64, 8, 2, 8, 32), ("i8", "bf16", 128, 7, 1, 16, 16), ("i8", "f32", 64, 4, 2, 8, 24)])
def test_serving_loop(fmt, dtype, d, hq, hkv, chunk, page):
    """A prompt moves into the cache, then tokens are decoded: append (own_len advances on the device), sparse decode,
    dense attention, and a gist step whenever a chunk completes.  Every output is checked against exact attention over
    the cache's values; the selection is the call's own."""
    B, L = 2, [chunk * 12, chunk * 7]
    steps, topk, n_max = chunk + 3, 4, 20
    p = Pool(B, hkv, d, chunk, page, chunk * 16, fmt)
    state = desc, pdesc, ws = p.desc(hq, dtype, n_max=n_max, topk=topk, exclude=False)
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dtype])  # noqa: E731
    gk, gv = rnd(B, hkv, n_max, d), rnd(B, hkv, n_max, d)
    own = torch.zeros(B, dtype=torch.int32, device="cuda")
    append(p, hq, own, L, dtype=dtype, rot=d, seed=1, state=state)
    n = torch.tensor([x // chunk for x in L], dtype=torch.int32, device="cuda")
    total = torch.tensor(L, dtype=torch.int32, device="cuda")
    out = torch.empty((B, hq, d), device="cuda")
    lse = torch.empty((B, hq), device="cuda")
    sel = torch.empty((B, hq, topk), dtype=torch.int32, device="cuda")
    o2, l2 = torch.empty((B, 1, hq, d), device="cuda"), torch.empty((B, 1, hq), device="cuda")
    s, grp = 1 / math.sqrt(d), hq // hkv
    for step in range(steps):
        pos = (total + total // chunk).to(torch.int32)
        r = append(p, hq, own, [1] * B, dtype=dtype, rot=d, seed=50 + step, state=state, n_gists=n, advance=True,
                   uniform=True, pos=pos)
        total += 1
        G.gsa_paged_decode(desc, pdesc, r["q_out"], gk, gv, *p_args(p), n, own, out, lse, sel, None, ws)
        G.gsa_paged_attend(desc, pdesc, 1, r["q_out"], *p_args(p), n, own, o2, l2, ws)
        assert (n * chunk + own).tolist() == total.tolist()
        for b in range(B):
            T, N = int(total[b]), int(n[b])
            k, v = p.rows("k", b, T), p.rows("v", b, T)
            for h in range(hq):
                q = r["q_out"][b, h].double()
                ids = sel[b, h].tolist()
                z = gk[b, h // grp, :N].double() @ q
                best = z.topk(min(topk, N)).values.min()
                assert all(float(z[m]) >= float(best) - 1e-4 * abs(float(best)) for m in ids if m >= 0)
                at = torch.tensor([x for m in ids if m >= 0 for x in range(m * chunk, (m + 1) * chunk)]
                                  + list(range(N * chunk, T)), device="cuda")
                kk = torch.cat([k[h // grp, at], gk[b, h // grp, :N].double()])
                vv = torch.cat([v[h // grp, at], gv[b, h // grp, :N].double()])
                check_row(out[b, h], lse[b, h], q, kk, vv, None, None, s, d, False, f"decode {step} {b} {h}",
                          prior=True)
                check_row(o2[b, 0, h], l2[b, 0, h], q, k[h // grp], v[h // grp], None, None, s, d, False,
                          f"dense {step} {b} {h}")
        if int(own[0]) == chunk:  # both sequences complete their chunks together
            q, kn, vn = rnd(B, hq, d), rnd(B, hkv, d), rnd(B, hkv, d)
            N0 = n.tolist()
            G.gsa_paged_gist_step(desc, pdesc, q, kn, vn, gk, gv, *p_args(p), n, own, out, lse, ws)
            assert n.tolist() == [x + 1 for x in N0] and own.tolist() == [0] * B
            for b in range(B):
                N = N0[b]
                assert torch.equal(gk[b, :, N], kn[b]) and torch.equal(gv[b, :, N], vn[b])
                k, v = (p.rows(x, b, int(total[b]))[:, N * chunk:] for x in "kv")
                for h in range(hq):
                    kk = torch.cat([k[h // grp], gk[b, h // grp, :N + 1].double()])
                    vv = torch.cat([v[h // grp], gv[b, h // grp, :N + 1].double()])
                    check_row(out[b, h], lse[b, h], q[b, h].double(), kk, vv, None, None, s, d, False, f"gist {b} {h}",
                              prior=True)
    assert G.gsa_workspace_status(ws) == 0


def p_args(p):
    return p.pages["k"], p.pages["v"], p.scales["k"], p.scales["v"], p.table


def test_decode_step_captured_and_replayed():
    """append + sparse decode as one graph: replayed steps give the bits of the same steps run one by one."""
    B, hq, hkv, d, chunk, page, topk, n_max = 2, 8, 2, 64, 8, 32, 3, 12
    runs = []
    for captured in (False, True):
        p = Pool(B, hkv, d, chunk, page, chunk * 12, "e4m3")
        state = desc, pdesc, ws = p.desc(hq, "bf16", n_max=n_max, topk=topk, exclude=False)
        g = torch.Generator(device="cuda").manual_seed(6)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        gk, gv = rnd(B, hkv, n_max, d), rnd(B, hkv, n_max, d)
        own = torch.zeros(B, dtype=torch.int32, device="cuda")
        append(p, hq, own, [chunk * 6, chunk * 3], rot=d, seed=1, state=state)
        n = torch.tensor([6, 3], dtype=torch.int32, device="cuda")
        q, k, v = torch.empty((B, hq, d), dtype=torch.bfloat16, device="cuda"), rnd(B, hkv, d), rnd(B, hkv, d)
        q_out, out = torch.empty_like(q), torch.empty((B, hq, d), device="cuda")
        inv = torch.tensor([0.5 ** i for i in range(d // 2)], device="cuda")
        ad = G.make_append_desc(B, d, False, True)

        def one():
            G.gsa_paged_append(desc, pdesc, ad, q, k, v, None, None, inv, p.table, n, own, *p.args()[1:], q_out, ws)
            G.gsa_paged_decode(desc, pdesc, q_out, gk, gv, *p_args(p), n, own, out, None, None, None, ws)

        outs = []
        if captured:
            side = torch.cuda.Stream()
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=side):
                one()
        for _ in range(5):
            for x, h in ((q, hq), (k, hkv), (v, hkv)):
                x.copy_(rnd(B, h, d))
            graph.replay() if captured else one()
            torch.cuda.synchronize()
            outs.append(out.clone())
        assert own.tolist() == [5, 5] and G.gsa_workspace_status(ws) == 0
        runs.append((outs, [p.pages[x].view(torch.uint8).clone() for x in "kv"], [p.scales[x].clone() for x in "kv"]))
    for a, b in zip(runs[0], runs[1]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_hgsa_selection_feeds_the_paged_unfold():
    """hgsa_select's prior and selection, then gsa_paged_unfold: the same outputs as hgsa_decode over an unpaged cache
    that holds the values of the codes (exactly representable there: e4m3 codes, power-of-two scales)."""
    B, hq, hkv, d, chunk, N, group = 2, 8, 2, 64, 8, 64, 8
    c = Cache([N * chunk + 5, N * chunk + 1], hkv, d, chunk, 32, "e4m3", seed=3)
    g = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, gk, gv, mk, mv = rnd(B, hq, d), rnd(B, hkv, N, d), rnd(B, hkv, N, d), rnd(B, hkv, 8, d), rnd(B, hkv, 8, d)
    n = torch.full((B,), N, dtype=torch.int32, device="cuda")
    own = torch.tensor([5, 1], dtype=torch.int32, device="cuda")
    hd = G.make_hdesc(group, 3, 8)
    t_max = c.cap
    desc = G.make_desc(B, hq, hkv, d, chunk, N, t_max, 6, False)
    pdesc = G.make_pdesc(G.GSA_E4M3, c.page, c.n_pages, c.max_pages)
    raw = {kv: torch.zeros((B, hkv, t_max, d), dtype=torch.bfloat16, device="cuda") for kv in "kv"}
    for kv in "kv":
        for b in range(B):
            raw[kv][b, :, :c.lens[b]] = c.rows(kv, b, c.lens[b]).to(torch.bfloat16)
            assert torch.equal(raw[kv][b, :, :c.lens[b]].double(), c.rows(kv, b, c.lens[b]))
    ws = torch.empty(G.gsa_workspace_bytes(desc, G.GSA_OP_HGSA, hd), dtype=torch.uint8, device="cuda")
    G.gsa_workspace_init(ws)
    mi = torch.empty((B, hq, 3), dtype=torch.int32, device="cuda")
    si, ss = torch.empty((B, hq, 6), dtype=torch.int32, device="cuda"), torch.empty((B, hq, 6), device="cuda")
    o, l, o2, l2 = (torch.empty(s, device="cuda") for s in ((B, hq, d), (B, hq), (B, hq, d), (B, hq)))
    G.hgsa_select(desc, hd, q, mk, mv, gk, gv, n, mi, si, ss, ws)
    G.gsa_paged_unfold(desc, pdesc, q, *c.args(), gv, n, own, si, ss, G.GSA_PRIOR_HGSA, o, l, ws)
    G.hgsa_decode(desc, hd, q, mk, mv, gk, gv, raw["k"], raw["v"], n, own, o2, l2, None, None, None, ws)
    torch.cuda.synchronize()
    # both are within 2e-3 / 2 of the same exact value (the unpaged path's own bound for bf16 inputs is 2e-3)
    assert float((o - o2).abs().max()) <= 4e-3 and float((l - l2).abs().max()) <= 4e-3
    assert G.gsa_workspace_status(ws) == 0
