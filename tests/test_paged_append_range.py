"""gsa_paged_append at the ends of its range: dims that no position turns, quotients next to a half step, more blocks than
CTAs, more heads than a warp takes at once."""
import math

import pytest
import torch

from _paged import block_scale
from test_paged_append import DT, Pool, check_rows, rotate, turn_slack

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


def plain_append(p, state, q, k, v, rot, inter, own):
    """One call for sequences of equal counts; returns the turned queries."""
    desc, pdesc, ws = state
    inv = torch.tensor([10000.0 ** (-2 * i / max(rot, 1)) for i in range(rot // 2)], dtype=torch.float32, device="cuda")
    q_out = torch.full_like(q, 77.0)
    G.gsa_paged_append(desc, pdesc, G.make_append_desc(k.shape[0], rot, inter), q, k, v, None, None,
                       inv if rot else None, p.table, None, own, *p.args()[1:], q_out, ws)
    assert G.gsa_workspace_status(ws) == 0
    return q_out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (128, 32), (128, 112), (64, 64)])
def test_dims_that_are_not_turned_keep_their_bits(dtype, inter, d, rot):
    """An inf, a NaN and zeros of both signs behind the turned dims: in the queries and in unquantised pages every
    value comes out as it went in, the neighbours' with it; values are never turned."""
    p = Pool(2, 2, d, 8, 16, 24, dtype)
    g = torch.Generator(device="cuda").manual_seed(d + rot)
    T = 26  # 13 tokens each
    q, k, v = (torch.randn((T, h, d), generator=g, device="cuda").to(DT[dtype]) for h in (6, 2, 2))
    for x in (q, k, v):
        first = 0 if x is v else rot
        for i in range(first, d, 3):
            x[i % T, i % x.shape[1], i] = (math.inf, -math.inf, -0.0, 0.0)[i % 4]
    q_out = plain_append(p, p.desc(6, dtype), q, k, v, rot, inter, torch.zeros(2, dtype=torch.int32, device="cuda"))
    word = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(q_out[..., rot:].view(word), q[..., rot:].view(word))
    assert torch.isfinite(q_out[..., :rot]).all()
    for b in range(2):
        at = torch.arange(13, device="cuda")
        pid = p.table[b].long()[at // 16]
        for kv, x, first in (("k", k, rot), ("v", v, 0)):
            got = p.pages[kv][pid, :, at % 16, first:]
            assert torch.equal(got.view(word), x[13 * b:13 * b + 13, :, first:].contiguous().view(word)), kv


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_int8_quotients_next_to_half_steps(dtype):
    """Values within a few fp32 steps of (k + 1/2) scales: a code is off by half a step of the exact quotient, plus the
    rounding of the quotient to fp32 (half of 2^-17 below 128; a reciprocal's would be up to three times that)."""
    d, blocks = 128, 64
    p = Pool(1, 1, d, 64, 64, 64 * blocks, "i8")
    g = torch.Generator(device="cuda").manual_seed(1)
    top = torch.exp(3 * torch.randn((blocks, 1, 1), generator=g, device="cuda"))  # each block's largest
    if dtype == "bf16":
        top = top.to(torch.bfloat16).float()
    s = (top.double() / 127).float()
    half = torch.randint(0, 127, (blocks, 64, d), generator=g, device="cuda") + 0.5
    x = (half.double() * s.double()).to(DT[dtype])
    if dtype == "f32":
        near = torch.randint(-2, 3, x.shape, generator=g, device="cuda", dtype=torch.int32)
        x = (x.view(torch.int32) + near).view(torch.float32)
    x = x * (1 - 2 * torch.randint(0, 2, x.shape, generator=g, device="cuda")).to(x.dtype)
    x[:, :1, :1] = top.to(x.dtype)
    x = x.clamp(-top.to(x.dtype), top.to(x.dtype)).view(blocks * 64, 1, d).contiguous()
    plain_append(p, p.desc(1, dtype), torch.zeros((len(x), 1, d), dtype=x.dtype, device="cuda"), x, x, 0, False,
                 torch.zeros(1, dtype=torch.int32, device="cuda"))
    for kv in "kv":
        pid = p.table[0].long()
        assert torch.equal(p.scales[kv][pid, 0, 0], s.flatten())
        code = p.pages[kv][pid, 0].double()
        off = (x.view(blocks, 64, d).double() / s.double() - code).abs()
        assert float(off.max()) <= 0.5 + 2.0 ** -18 + 2.0 ** -40, float(off.max()) - 0.5


MANY = [
    # fmt, dtype, d, hq, hkv, chunk, page, held, new, rot, inter: thousands of blocks, so a CTA takes several
    ("e4m3", "bf16", 64, 32, 2, 8, 64, [5, 0, 3, 1000], [20000, 1, 77, 4099], 64, False),
    ("i8", "bf16", 128, 28, 4, 8, 32, [0, 13, 7], [9000, 2, 7001], 128, True),
    ("i8", "f32", 64, 20, 4, 4, 20, [2, 0], [11, 7000], 32, False),
    ("e4m3", "f32", 128, 9, 1, 7, 21, [6, 0, 0], [6000, 1300, 1], 112, True),
    ("bf16", "bf16", 64, 17, 17, 16, 48, [0, 15], [100, 15000], 16, False),
    ("e4m3", "bf16", 64, 20, 2, 1, 1, [0, 0], [1501, 900], 48, True),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: f"{c[0]}_{c[1]}_d{c[2]}_{c[3]}x{c[4]}_c{c[5]}_rot{c[9]}")
def test_prompts_of_thousands_of_blocks(case):
    """Every query, key and value of long ragged prompts, the first of them behind part-filled blocks."""
    fmt, dtype, d, hq, hkv, chunk, page, held, new, rot, inter = case
    B = len(held)
    p = Pool(B, hkv, d, chunk, page, max(a + b for a, b in zip(held, new)), fmt, seed=hq)
    desc, pdesc, ws = p.desc(hq, dtype)
    inv = torch.tensor([10000.0 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float32, device="cuda")
    own = torch.zeros(B, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(hq + d)
    for start, n in (([0] * B, held), (held, new)):
        T = sum(n)
        q, k, v = (torch.randn((T, h, d), generator=g, device="cuda").to(DT[dtype]) for h in (hq, hkv, hkv))
        cu = torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32, device="cuda")
        q_out = torch.full_like(q, 77.0)
        G.gsa_paged_append(desc, pdesc, G.make_append_desc(T, rot, inter, True), q, k, v, cu, None, inv, p.table, None,
                           own, *p.args()[1:], q_out, ws)
    assert own.tolist() == [a + b for a, b in zip(held, new)] and G.gsa_workspace_status(ws) == 0
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(new, device="cuda"))
    row = torch.arange(T, device="cuda") - cu.long()[seq] + torch.tensor(held, device="cuda")[seq]
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for lo in range(0, T, 4096):  # in pieces: 64-bit copies
        sl = slice(lo, lo + 4096)
        want = rotate(q[sl], row[sl], inv, inter)
        lim = want.abs() * half * (1 + 2.0 ** -8) + turn_slack(q[sl], rot, inter)
        assert bool(((q_out[sl].double() - want).abs() <= lim).all()), f"queries from token {lo}"
    pid, off = p.table.long()[seq, row // page], row % page
    for kv, x, slack in (("k", rotate(k, row, inv, inter), turn_slack(k, rot, inter)),
                         ("v", v.double(), torch.zeros((T, hkv, d), dtype=torch.float64, device="cuda"))):
        got, s = p.pages[kv].view(torch.uint8 if fmt == "e4m3" else p.pages[kv].dtype)[pid, :, off], None
        got = got.view(p.pages[kv].dtype).double()
        if p.scales[kv] is not None:
            s = p.scales[kv][pid, :, off // chunk].double()[..., None]
            got = got * s
        check_rows(got, x, slack, s, fmt, 1, kv)
        if s is None:
            continue
        # scales of the blocks that this call began
        block = torch.cumsum(((row % chunk == 0) | (row == torch.tensor(held, device="cuda")[seq])).long(), 0) - 1
        top = torch.zeros((int(block[-1]) + 1, hkv), dtype=torch.float64, device="cuda")
        top.index_reduce_(0, block, x.abs().amax(-1), "amax")
        want = block_scale(top, fmt)[block]
        begun = (row - row % chunk >= torch.tensor(held, device="cuda")[seq])[:, None]
        # (int8: the turned maximum's error and the division; e4m3: the same power of two, unless the maximum is
        # within that error of 448 scales)
        near = (top / block_scale(top, fmt) > 448 * (1 - 2.0 ** -20))[block] if fmt == "e4m3" else torch.zeros_like(begun)
        lim = want * (2.0 ** -20 if fmt == "i8" else 0)
        assert bool((((s[..., 0] - want).abs() <= lim) | ~begun | near).all()), f"scales of {kv}"
