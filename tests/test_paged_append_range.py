"""gsa_paged_append at the ends of its range: dims that no position turns, quotients next to a half step."""
import math

import pytest
import torch

from test_paged_append import DT, Pool

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
