"""Cases for the paged 8-bit raw-token cache: appending rotated keys and values, attention over the whole cache and
selective unfolding from it.

Each case is one call as a serving loop makes it.  `run` computes the call's plain form in elementary torch operations;
with `own` set it makes the call through the package.  A sequence's rows lie in pages of a shared pool
[pages, kv heads, rows of a page, d], found through a page table; the codes of a block of `chunk` rows and one kv head
share one fp32 scale.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn, "bf16": torch.bfloat16, "f32": torch.float32}
BASE = 500000.0  # base of the rotation's frequencies


# ------------------------------------------------------------------ cases
def listed():
    def case(name, op, **kw):
        c = dict(name=name, op=op, batch=1, hq=32, hkv=8, d=64, chunk=8, page=64, cache="e4m3", dtype="bf16", out="bf16",
                 len=1000, ragged=False, n_q=1, topk=0, n_new=1, rot=64, inter=False)
        c.update(kw)
        return c

    return [
        # one token of one sequence joins a part-filled block (the decode step of a chat): latency
        case("append_step_1", "append", len=1003),
        # one token for each of 64 sequences of different lengths, 128-dim heads at 16x compression
        case("append_step_64", "append", batch=64, hq=28, hkv=4, d=128, chunk=16, page=128, len=20000, ragged=True,
             rot=128),
        # a prefilled 32K prompt moves into the cache, queries rotated on the way
        case("append_prompt_32k", "append", batch=1, len=0, n_new=32768),
        # uneven prompts behind cached prefixes, unquantised pages, interleaved pairs, part of the head rotated
        case("append_ragged_f32", "append", batch=7, hq=8, hkv=2, d=128, chunk=24, page=48, cache="f32", dtype="f32",
             len=700, ragged=True, n_new=1291, rot=32, inter=True),
        # a short conversation's decode step: latency
        case("attend_short", "attend", len=200),
        # dense attention at the 1B-class decode shape: 16 x 32K tokens, 8-token blocks
        case("attend_16x32k", "attend", batch=16, len=32771, out="f32"),
        # dense attention at the 7B-class decode shape: 4 x 128K tokens, int8 codes
        case("attend_4x128k_i8", "attend", batch=4, hq=28, hkv=4, d=128, chunk=16, page=128, cache="i8", len=131072),
        # a ragged batch checking 4 drafted tokens each, fp32 queries, pages that end inside a tile
        case("attend_ragged_draft", "attend", batch=37, hq=16, hkv=4, d=128, chunk=24, page=24, cache="i8", dtype="f32",
             out="f32", len=9001, ragged=True, n_q=4),
        # a single-head fp32 step, top-8 of 256 chunks: latency
        case("unfold_tiny_f32", "unfold", hq=1, hkv=1, chunk=16, page=64, cache="i8", dtype="f32", out="f32", len=4099,
             topk=8),
        # the 1B-class decode shape: top-64 of 4096 8-token chunks, 16 sequences
        case("unfold_16x32k", "unfold", batch=16, len=32771, topk=64),
        # the 7B-class decode shape: top-128 of 8192 16-token chunks, 4 sequences
        case("unfold_4x128k_i8", "unfold", batch=4, hq=28, hkv=4, d=128, chunk=16, page=128, cache="i8", len=131077,
             topk=128, out="f32"),
        # 32x compression over 512K tokens: top-64 chunks of 32 tokens
        case("unfold_2x512k", "unfold", batch=2, hq=32, hkv=8, d=128, chunk=32, page=256, len=524288, topk=64),
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["append", "attend", "unfold"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 7, 8, 16]) if op != "append" else rng.choice([1, 4, 7])
    chunk = rng.choice([4, 7, 8, 16, 24, 32, 64])
    page = chunk * rng.choice([1, 2, 3, 4, 8, 16])
    c = dict(op=op, batch=log_int(1, 64), hq=hkv * group, hkv=hkv, d=d, chunk=chunk, page=page, cache="e4m3", dtype="bf16",
             out=rng.choice(["bf16", "f32"]), len=log_int(1, 131072), ragged=rng.random() < 0.5, n_q=1, topk=0, n_new=1,
             rot=rng.choice([16, 32, d]), inter=rng.random() < 0.3)
    if op == "append":
        if rng.random() < 0.5:
            c["n_new"] = log_int(1, 16384)
        if rng.random() < 0.3:
            c["cache"] = c["dtype"] = rng.choice(["bf16", "f32"])
        # no more bytes than the largest listed append; the pool stays within a few GB
        token = hkv * d * DT[c["dtype"]].itemsize * (2 * group + 4)
        c["batch"] = max(1, min(c["batch"], (1 << 28) // (c["n_new"] * token)))
        c["n_new"] = max(1, min(c["n_new"], (1 << 28) // (c["batch"] * token)))
        c["len"] = min(c["len"], 32768, (1 << 29) // (c["batch"] * hkv * d))
    else:
        c["cache"] = rng.choice(["i8", "e4m3"])
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        if op == "attend":
            c["n_q"] = rng.choice([1, 1, 1, 2, 5])
            c["batch"] = max(1, min(c["batch"], (1 << 28) // (c["len"] * hkv * d)))
            c["len"] = max(c["n_q"], min(c["len"], (1 << 28) // (c["batch"] * hkv * d * ((c["n_q"] * group + 15) // 16))))
        else:
            c["topk"] = log_int(1, 256)
            c["batch"] = max(1, min(c["batch"], (1 << 28) // (c["len"] * hkv * d)))
            c["batch"] = max(1, min(c["batch"], (1 << 24) // (c["hq"] * c["topk"] * chunk * d) or 1))
    return c


def _lens(c):
    """Rows already cached in each sequence, and the tokens that join (append): fixed by the case alone."""
    B, n = c["batch"], c["len"]
    rng = random.Random(B * 7919 + n)
    if not c["ragged"]:
        lens = [n] * B
    else:
        lo = max(c["n_q"] if c["op"] == "attend" else 0, n // 50)
        lens = [int(lo + (n - lo) * ((i + 0.5) / B) ** 2) for i in range(B)]
        rng.shuffle(lens)
    if c["op"] != "append":
        return lens, [0] * B
    new = [c["n_new"]] * B
    if c["ragged"] and c["n_new"] > 1:
        new = [max(1, int(c["n_new"] * 2 * (i + 0.5) / B)) for i in range(B)]
        rng.shuffle(new)
    return lens, new


def work(case):
    c = case
    lens, new = _lens(c)
    e, o = DT[c["dtype"]].itemsize, DT[c["out"]].itemsize
    code = CODE[c["cache"]].itemsize
    scaled = 8 / c["chunk"] if code == 1 else 0
    if c["op"] == "append":
        T = sum(new)
        return dict(bytes=T * c["d"] * (2 * c["hq"] * e + 2 * c["hkv"] * (e + code)) + T * c["hkv"] * scaled + 4 * T,
                    flops=3 * T * c["rot"] * (c["hq"] + c["hkv"]))
    if c["op"] == "attend":
        rows = sum(lens)
        return dict(bytes=rows * c["hkv"] * (2 * c["d"] + scaled) + c["batch"] * c["n_q"] * c["hq"] * (c["d"] * (e + o) + 4),
                    flops=4 * rows * c["hq"] * c["n_q"] * c["d"])
    rows = sum(min(c["topk"], n // c["chunk"]) * c["chunk"] + n % c["chunk"] for n in lens)
    gists = sum(min(c["topk"], n // c["chunk"]) for n in lens)
    return dict(bytes=c["hq"] * (rows * (2 * c["d"] + scaled) + gists * (c["d"] * e + 8) + c["batch"] * (c["d"] * (e + o) + 4)),
                flops=4 * c["hq"] * c["d"] * (rows + gists / 2))


# ------------------------------------------------------------------ inputs
def _block_scale(amax, cache):
    """The scale of a block whose largest magnitude is amax (fp32)."""
    if cache == "i8":
        s = amax / 127.0
    else:
        m, e = torch.frexp(amax)
        s = torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).int())
    return torch.where(amax < 2.0 ** -100, torch.zeros_like(s), s)


def _code(x, cache):
    """x (already divided by its scale) in the cache's type."""
    if cache == "i8":
        return torch.clamp(torch.round(x), -127, 127).to(torch.int8)
    return x.to(CODE[cache])


def _pool(rows, c, g, dev):
    """A pool of `rows` blocks of random rows, quantised: pages [blocks, hkv, chunk, d] and scales."""
    std = torch.exp(0.5 * torch.randn((1, c["hkv"], 1, 1), generator=g, device=dev))
    shape = (rows, c["hkv"], c["chunk"], c["d"])
    codes = torch.empty(shape, dtype=CODE[c["cache"]], device=dev)
    if codes.element_size() > 1:
        codes.copy_(torch.randn(shape, generator=g, device=dev) * std)
        return codes, None
    scale = torch.empty(shape[:2], dtype=torch.float32, device=dev)
    step = max(1, (1 << 26) // (c["hkv"] * c["chunk"] * c["d"]))
    for i in range(0, rows, step):
        x = torch.randn((min(step, rows - i),) + shape[1:], generator=g, device=dev) * std
        s = _block_scale(x.abs().amax((2, 3)), c["cache"])
        codes[i:i + step] = _code(x / s[:, :, None, None], c["cache"])
        scale[i:i + step] = s
    return codes, scale


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    lens, new = _lens(c)
    B, chunk, page, hq, hkv, d = c["batch"], c["chunk"], c["page"], c["hq"], c["hkv"], c["d"]
    dt = DT[c["dtype"]]
    cap = max(a + b for a, b in zip(lens, new))
    max_pages = max(1, -(-cap // page))
    # every sequence has the pages that its rows need, in no order; two pages of the pool are nobody's
    need = [-(-(a + b) // page) for a, b in zip(lens, new)]
    n_pages = sum(need) + 2
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    taken = torch.tensor(need, device=dev)
    first = torch.cumsum(taken, 0) - taken
    slot = torch.arange(max_pages, device=dev)[None, :]
    table = torch.where(slot < taken[:, None], order[(first[:, None] + slot).clamp_(max=n_pages - 1)],
                        torch.full((), 0, dtype=torch.int32, device=dev)).contiguous()
    s = dict(case=c, lens=lens, new=new, table=table, n_pages=n_pages, max_pages=max_pages, cap=cap,
             own_len=torch.tensor(lens, dtype=torch.int32, device=dev))
    for kv in "kv":
        codes, scale = _pool(n_pages * (page // chunk), c, g, dev)
        codes = codes.view(n_pages, page // chunk, hkv, chunk, d).transpose(1, 2)
        s[kv + "_pages"] = codes.reshape(n_pages, hkv, page, d)
        s[kv + "_scale"] = None if scale is None else scale.view(n_pages, page // chunk, hkv).transpose(1, 2).contiguous()
        del codes, scale

    def rand(shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dt)

    if c["op"] == "append":
        T = sum(new)
        s.update(q=rand((T, hq, d)), k=rand((T, hkv, d), 1.2), v=rand((T, hkv, d)),
                 cu=torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device=dev),
                 q_out=torch.empty((T, hq, d), dtype=dt, device=dev),
                 inv_freq=torch.tensor([BASE ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)], dtype=torch.float32,
                                       device=dev))
        tok = torch.arange(T, device=dev)
        seq = torch.searchsorted(s["cu"][1:].long(), tok, right=True)
        # positions count each finished chunk's gist token, as the model that reads this cache does
        row = tok - s["cu"][seq] + s["own_len"][seq]
        s["pos"] = (row + row // chunk).to(torch.int32)
    elif c["op"] == "attend":
        s["q"] = rand((B, c["n_q"], hq, d))
    else:
        k = c["topk"]
        n = torch.tensor([x // chunk for x in lens], device=dev)
        n_max = max(1, cap // chunk)
        s["n_gists"], s["n_max"] = n.to(torch.int32), n_max
        s["own_len"] = torch.tensor([x % chunk for x in lens], dtype=torch.int32, device=dev)
        s["q"] = rand((B, hq, d))
        s["gist_v"] = rand((B, hkv, n_max, d))
        # k different completed chunks for each query head, ascending, -1 behind them; scores of chunks that were chosen
        # for being high
        key = torch.rand((B, hq, max(n_max, k)), generator=g, device=dev)
        key.masked_fill_(torch.arange(max(n_max, k), device=dev) >= n[:, None, None], 2.0)
        val, idx = key.topk(k, largest=False)
        idx = torch.where(val > 1.5, torch.full_like(idx, 1 << 30), idx).sort(-1).values
        s["sel_idx"] = torch.where(idx >= 1 << 30, torch.full_like(idx, -1), idx).to(torch.int32).contiguous()
        s["sel_score"] = torch.where(s["sel_idx"] >= 0, 2.0 + torch.randn((B, hq, k), generator=g, device=dev),
                                     torch.full((), -math.inf, device=dev)).contiguous()
    return s


# ------------------------------------------------------------------ plain form
def _softmax_av(z, v):
    """Rows of logits z [.., R, T] (-inf: left out) and values v [.., T, d]: the weighted mean and ln of the sum."""
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(z - m)
    tot = p.sum(-1, keepdim=True)
    return torch.where(tot > 0, (p @ v) / tot, torch.zeros((), device=z.device)), (m + torch.log(tot)).squeeze(-1)


def _codes(pages, at):
    """pages[at] (the 8-bit types are indexed as bytes)."""
    return pages.view(torch.uint8)[at].view(pages.dtype)


def _attend(s):
    c = s["case"]
    B, hkv, d, G, nq = c["batch"], c["hkv"], c["d"], c["hq"] // c["hkv"], c["n_q"]
    T = s["max_pages"] * c["page"]

    def rows(kv):
        x = _codes(s[kv + "_pages"], s["table"].long()).float()
        x = x.view(B, -1, hkv, c["page"] // c["chunk"], c["chunk"], d) * s[kv + "_scale"][s["table"].long()][..., None, None]
        return x.view(B, -1, hkv, c["page"], d).transpose(1, 2).reshape(B, hkv, T, d)

    q = s["q"].float().view(B, nq, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, nq * G, d)
    z = (q @ rows("k").transpose(-1, -2)).view(B, hkv, nq, G, T) / math.sqrt(d)
    end = s["own_len"][:, None] - (nq - 1) + torch.arange(nq, device=z.device)
    live = torch.arange(T, device=z.device) < end[:, :, None]
    z = torch.where(live[:, None, :, None, :], z, torch.full((), -math.inf, device=z.device))
    out, lse = _softmax_av(z.view(B, hkv, nq * G, T), rows("v"))
    out = out.view(B, hkv, nq, G, d).permute(0, 2, 1, 3, 4).reshape(B, nq, hkv * G, d)
    return out.to(DT[c["out"]]), lse.view(B, hkv, nq, G).transpose(1, 2).reshape(B, nq, hkv * G)


def _unfold(s):
    c = s["case"]
    B, hq, hkv, d, chunk, page = c["batch"], c["hq"], c["hkv"], c["d"], c["chunk"], c["page"]
    dev = s["q"].device
    sel = s["sel_idx"].long()
    raw = sel[..., None] * chunk + torch.arange(chunk, device=dev)
    raw = torch.where(sel[..., None] >= 0, raw, torch.full((), -1, device=dev)).flatten(2)
    tail = torch.arange(chunk, device=dev)
    tail = torch.where(tail < s["own_len"][:, None], s["n_gists"][:, None] * chunk + tail, torch.full((), -1, device=dev))
    raw = torch.cat([raw, tail[:, None, :].expand(B, hq, chunk)], -1)
    live, raw = raw >= 0, raw.clamp(min=0)
    pid = s["table"].long().gather(1, (raw // page).view(B, -1).clamp(max=s["max_pages"] - 1)).view_as(raw)
    head = (torch.arange(hq, device=dev) // (hq // hkv))[None, :, None]

    def rows(kv):
        x = _codes(s[kv + "_pages"], (pid, head, raw % page)).float()
        return x * s[kv + "_scale"][pid, head, (raw % page) // chunk][..., None]

    z = (rows("k") @ s["q"].float()[..., None]).squeeze(-1) / math.sqrt(d)
    z = torch.where(live, z, torch.full((), -math.inf, device=dev))
    gv = s["gist_v"][torch.arange(B, device=dev)[:, None, None], head, sel.clamp(min=0)].float()
    z = torch.cat([z, torch.where(sel >= 0, s["sel_score"], torch.full((), -math.inf, device=dev))], -1)
    out, lse = _softmax_av(z[:, :, None, :], torch.cat([rows("v"), gv], 2))
    return out.squeeze(2).to(DT[c["out"]]), lse.squeeze(2)


def _rotate(x, s):
    """x [T, heads, d] with its first rot dims turned by position; angles in 64 bits, the rest in 32."""
    c = s["case"]
    rot = c["rot"]
    ang = s["pos"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["inter"] else (y[..., :rot // 2], y[..., rot // 2:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if c["inter"] else torch.cat([ra, rb], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _append(s):
    c = s["case"]
    chunk, page, hkv, d = c["chunk"], c["page"], c["hkv"], c["d"]
    dev = s["k"].device
    T = s["k"].shape[0]
    tok = torch.arange(T, device=dev)
    seq = torch.searchsorted(s["cu"][1:].long(), tok, right=True)
    row = tok - s["cu"].long()[seq] + s["own_len"].long()[seq]
    pid = s["table"].long()[seq, row // page]
    off = row % page
    s["q_out"].copy_(_rotate(s["q"], s))
    head = torch.arange(hkv, device=dev)
    # the first new token of each block, and each token's block in that list
    lead = (tok == s["cu"].long()[seq]) | (row % chunk == 0)
    block = torch.cumsum(lead.long(), 0) - 1
    bp, bo = pid[lead][:, None], (off // chunk)[lead][:, None]
    held = (row % chunk)[lead]
    for kv, x in (("k", _rotate(s["k"], s)), ("v", s["v"].float())):
        pages, scale = s[kv + "_pages"], s[kv + "_scale"]
        if scale is None:
            pages[pid[:, None], head, off[:, None]] = x.to(pages.dtype)
            continue
        amax = torch.zeros((bp.shape[0], hkv), device=dev).index_reduce(0, block, x.abs().amax(-1), "amax")
        old = torch.where(held[:, None] > 0, scale[bp, head, bo], torch.zeros((), device=dev))
        s_new = torch.maximum(old, _block_scale(amax, c["cache"]))
        scale[bp, head, bo] = s_new
        # rows that the block held already, at the new scale
        r = torch.arange(chunk, device=dev)
        bytes_ = pages.view(torch.uint8)
        at = (bp[:, :, None], head[:, None], bo[:, :, None] * chunk + r)
        rows = bytes_[at].view(pages.dtype).float() * torch.where(s_new > 0, old / s_new, torch.zeros((), device=dev))[..., None, None]
        keep = (r < held[:, None])[:, None, :, None]
        bytes_[at] = torch.where(keep, _code(rows, c["cache"]).view(torch.uint8), bytes_[at])
        div = torch.where(s_new > 0, s_new, torch.ones((), device=dev))[block][..., None]
        bytes_[pid[:, None], head, off[:, None]] = _code(x / div, c["cache"]).view(torch.uint8)
    return tuple(t for t in (s["q_out"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]) if t is not None)


# ------------------------------------------------------------------ the package's calls
def _plan(s):
    """Descriptors, workspace and output buffers: made once for a shape, as a serving loop does."""
    import long_context_gsa_b200 as G
    c = s["case"]
    dt = {"bf16": G.GSA_BF16, "f32": G.GSA_F32, "i8": G.GSA_I8, "e4m3": G.GSA_E4M3}
    dev, B, hq, d = "cuda", c["batch"], c["hq"], c["d"]
    desc = G.make_desc(B, hq, c["hkv"], d, c["chunk"], s.get("n_max", 1), s["cap"], c["topk"], True, 0.0, dt[c["dtype"]],
                       dt[c["out"]])
    p = dict(G=G, desc=desc, pdesc=G.make_pdesc(dt[c["cache"]], c["page"], s["n_pages"], s["max_pages"]))
    p["ws"] = torch.empty(G.gsa_workspace_bytes(desc, G.GSA_OP_PAGED), dtype=torch.uint8, device=dev)
    G.gsa_workspace_init(p["ws"])
    if c["op"] == "append":
        p["adesc"] = G.make_append_desc(s["k"].shape[0], c["rot"], c["inter"])
    else:
        shape = (B, c["n_q"], hq) if c["op"] == "attend" else (B, hq)
        p["out"] = torch.empty(shape + (d,), dtype=DT[c["out"]], device=dev)
        p["lse"] = torch.empty(shape, dtype=torch.float32, device=dev)
    return p


def _own_run(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    p, c = s["plan"], s["case"]
    G = p["G"]
    if c["op"] == "append":
        G.gsa_paged_append(p["desc"], p["pdesc"], p["adesc"], s["q"], s["k"], s["v"], s["cu"], s["pos"], s["inv_freq"],
                           s["table"], None, s["own_len"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                           s["q_out"], p["ws"])
        return tuple(t for t in (s["q_out"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]) if t is not None)
    if c["op"] == "attend":
        G.gsa_paged_attend(p["desc"], p["pdesc"], c["n_q"], s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                           s["table"], None, s["own_len"], p["out"], p["lse"], p["ws"])
    else:
        G.gsa_paged_unfold(p["desc"], p["pdesc"], s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                           s["table"], s["gist_v"], s["n_gists"], s["own_len"], s["sel_idx"], s["sel_score"],
                           G.GSA_PRIOR_NONE, p["out"], p["lse"], p["ws"])
    return p["out"], p["lse"]


def run(state):
    if own:
        return _own_run(state)
    return {"append": _append, "attend": _attend, "unfold": _unfold}[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits
def _deq64(codes, scale, chunk):
    """[hkv, rows, d] codes and [hkv, blocks] scales in 64 bits."""
    return codes.double() * scale.double().repeat_interleave(chunk, -1)[:, :, None]


def _attn64(q, k, v, extra_z=None, extra_v=None):
    z = k @ q / math.sqrt(q.shape[-1])
    if extra_z is not None:
        z, v = torch.cat([z, extra_z.double()]), torch.cat([v, extra_v.double()])
    if z.numel() == 0:
        return torch.zeros_like(q), q.new_full((), -math.inf)
    lse = torch.logsumexp(z, 0)
    return torch.exp(z - lse) @ v, lse


def exact(case, seed):
    c = case
    if work(c)["flops"] > 4e11 or c["batch"] * c["hq"] * max(1, c["topk"] > 0) > 4096:
        return None
    s = prepare(case, seed)
    chunk, page, hkv, d, G = c["chunk"], c["page"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    dev = s["table"].device
    if c["op"] == "append":
        return _exact_append(s)
    nq = c["n_q"]
    shape = (c["batch"], nq, c["hq"]) if c["op"] == "attend" else (c["batch"], c["hq"])
    out = torch.zeros(shape + (d,), dtype=torch.float64, device=dev)
    lse = torch.full(shape, -math.inf, dtype=torch.float64, device=dev)
    for b in range(c["batch"]):
        n = s["lens"][b]
        ids = s["table"][b, :-(-n // page)].long()
        k, v = (_deq64(s[x + "_pages"][ids].transpose(0, 1).reshape(hkv, -1, d),
                       s[x + "_scale"][ids].transpose(0, 1).reshape(hkv, -1), chunk) for x in "kv")
        if c["op"] == "attend":
            for i in range(nq):
                end = max(0, n - (nq - 1) + i)
                if end == 0:
                    continue
                q = s["q"][b, i].double().view(hkv, G, d)
                z = torch.einsum("hgd,htd->hgt", q, k[:, :end]) / math.sqrt(d)
                tot = torch.logsumexp(z, -1)
                lse[b, i] = tot.reshape(-1)
                out[b, i] = torch.einsum("hgt,htd->hgd", torch.exp(z - tot[..., None]), v[:, :end]).reshape(-1, d)
            continue
        done = n - n % chunk
        sel = s["sel_idx"][b].cpu().tolist()
        for h in range(c["hq"]):
            ch = torch.tensor([m for m in sel[h] if m >= 0], dtype=torch.long, device=dev)
            at = torch.cat([(ch[:, None] * chunk + torch.arange(chunk, device=dev)).flatten(),
                            torch.arange(done, n, device=dev)])
            e = s["sel_score"][b, h, :len(ch)], s["gist_v"][b, h // G, ch]
            out[b, h], lse[b, h] = _attn64(s["q"][b, h].double(), k[h // G, at], v[h // G, at], *e)
    return out, lse


def _exact_append(s):
    """Each sequence's touched pages as one dense run of rows, its new rows put behind the held ones."""
    c = s["case"]
    chunk, page, hkv, d, rot = c["chunk"], c["page"], c["hkv"], c["d"], c["rot"]
    if c["cache"] == "i8":
        return None
    dev = s["k"].device
    ang = s["pos"].double()[:, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(ang), ang)[:, None, :]

    def rotate(x):
        y = x.double().clone()
        ia = torch.arange(0, rot, 2, device=dev) if c["inter"] else torch.arange(rot // 2, device=dev)
        ib = ia + (1 if c["inter"] else rot // 2)
        w = torch.complex(y[..., ia], y[..., ib]) * turn
        y[..., ia], y[..., ib] = w.real, w.imag
        return y

    def e4m3(x):
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(x.abs().clamp(min=1e-300))), min=-6.0) - 3.0)
        return torch.round(x / step) * step

    res = {"q": rotate(s["q"])}
    for kv, x in (("k", rotate(s["k"])), ("v", s["v"].double())):
        pages = s[kv + "_pages"].double()
        scale = None if s[kv + "_scale"] is None else s[kv + "_scale"].double()
        at = 0
        for b, (n, t) in enumerate(zip(s["lens"], s["new"])):
            new, at = x[at:at + t].transpose(0, 1), at + t
            first = n // page
            ids = s["table"][b, first:-(-(n + t) // page)].long()
            mine = pages[ids].transpose(0, 1).reshape(hkv, -1, d)  # rows first*page ..
            r0 = n - first * page
            if scale is None:
                mine[:, r0:r0 + t] = new
            else:
                nb = mine.shape[1] // chunk
                sc = scale[ids].transpose(0, 1).reshape(hkv, nb)
                b0, b1 = r0 // chunk, -(-(r0 + t) // chunk)
                val = torch.zeros((hkv, (b1 - b0) * chunk, d), dtype=torch.float64, device=dev)
                lo = r0 - b0 * chunk
                val[:, lo:lo + t] = new
                amax = val.view(hkv, b1 - b0, chunk * d).abs().amax(-1)
                want = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
                want = torch.where(amax < 2.0 ** -100, torch.zeros_like(want), want)
                was = sc[:, b0:b1].clone()
                was[:, (1 if lo else 0):] = 0.0
                want = torch.maximum(want, was)
                if lo:
                    val[:, :lo] = mine[:, b0 * chunk:r0] * was[:, :1, None]
                sc[:, b0:b1] = want
                div = torch.where(want > 0, want, torch.ones_like(want)).repeat_interleave(chunk, 1)[..., None]
                mine[:, b0 * chunk:r0 + t] = e4m3(val[:, :lo + t] / div[:, :lo + t])
                scale[ids] = sc.view(hkv, len(ids), -1).transpose(0, 1)
            pages[ids] = mine.view(hkv, len(ids), page, d).transpose(0, 1)
        res[kv], res[kv + "s"] = pages, scale
    return tuple(t for t in (res["q"], res["k"], res["v"], res["ks"], res["vs"]) if t is not None)
