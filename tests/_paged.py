"""A paged 8-bit raw-token cache in plain torch, 64 bits: building one, reading
its rows and attending them.  Shares no code with the library."""
import math

import torch

CODE = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn, "bf16": torch.bfloat16, "f32": torch.float32}


def block_scale(amax, fmt):
    """Scale of a block whose largest magnitude is amax (float64)."""
    if fmt == "i8":
        s = amax / 127.0
    else:
        s = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
    return torch.where(amax < 2.0 ** -100, torch.zeros_like(s), s)


def encode(x, s, fmt):
    y = torch.where(s > 0, x / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x))
    if fmt == "i8":
        return torch.clamp(torch.round(y), -127, 127).to(torch.int8)
    return y.to(torch.float32).to(torch.float8_e4m3fn)


class Cache:
    """A pool with a shuffled page table.  Rows and pages that hold nothing are filled with garbage: NaN codes
    (e4m3) or -128 (int8), NaN scales in unused blocks."""

    def __init__(self, lens, hkv, d, chunk, page, fmt, *, spare=0, seed=0, dev="cuda", std=1.0, share=None):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        self.lens, self.hkv, self.d, self.chunk, self.page, self.fmt = list(lens), hkv, d, chunk, page, fmt
        B = len(lens)
        self.cap = max(1, max(lens) + spare)
        self.max_pages = -(-self.cap // page)
        self.n_pages = B * self.max_pages + 3
        perm = torch.randperm(self.n_pages, generator=g, device=dev)[:B * self.max_pages]
        self.table = perm.view(B, self.max_pages).to(torch.int32).contiguous()
        if share is not None:  # sequence 1.. read sequence 0's first `share` pages
            self.table[1:, :share] = self.table[:1, :share]
        nb = page // chunk
        self.pages, self.scales = {}, {}
        for kv in "kv":
            rows = torch.randn((self.n_pages, hkv, page, d), generator=g, device=dev, dtype=torch.float64)
            rows *= std * torch.exp(0.7 * torch.randn((self.n_pages, hkv, 1, 1), generator=g, device=dev,
                                                      dtype=torch.float64))
            if fmt in ("bf16", "f32"):
                self.pages[kv], self.scales[kv] = rows.to(CODE[fmt]), None
                continue
            blocks = rows.view(self.n_pages, hkv, nb, chunk, d)
            s = block_scale(blocks.abs().amax((3, 4)), fmt).float()
            codes = encode(blocks, s.double()[..., None, None], fmt).view(self.n_pages, hkv, page, d)
            byte = codes.view(torch.uint8)
            used = torch.zeros((self.n_pages, page), dtype=torch.bool, device=dev)
            for b, n in enumerate(lens):
                for p in range(self.max_pages):
                    used[int(self.table[b, p]), :max(0, min(page, n - p * page))] = True
            byte[(~used)[:, None, :].expand(-1, hkv, -1)] = 0x7F if fmt == "e4m3" else 0x80
            live = used.view(self.n_pages, nb, chunk).any(-1)
            s[(~live)[:, None, :].expand(-1, hkv, -1)] = float("nan")
            self.pages[kv], self.scales[kv] = codes, s.contiguous()

    def rows(self, kv, b, n):
        """The first n raw rows of sequence b in float64: [hkv, n, d]."""
        out = []
        for p in range(-(-n // self.page)):
            pid = int(self.table[b, p])
            x = self.pages[kv][pid].double()
            if self.scales[kv] is not None:
                x = x * self.scales[kv][pid].double().repeat_interleave(self.chunk, -1)[..., None]
            out.append(x)
        if not out:
            return torch.zeros((self.hkv, 0, self.d), dtype=torch.float64, device=self.table.device)
        return torch.cat(out, 1)[:, :n]

    def args(self):
        return self.pages["k"], self.pages["v"], self.scales["k"], self.scales["v"], self.table


def softmax_av(z, v):
    """Exact attention of one row: logits z [n], values v [n, d] -> (out, lse)."""
    if z.numel() == 0:
        return torch.zeros(v.shape[-1], dtype=torch.float64, device=v.device), torch.tensor(-math.inf)
    lse = torch.logsumexp(z, 0)
    return torch.exp(z - lse) @ v, lse


def logit_error(d, reach, floor):
    """How far a base-2 logit may be off.

    reach: the largest log2(e) * scale * sum_i |q_i k_i| of an attended row; floor: the same with every |q_i| replaced
    by the row's largest.  The products of the operands' digits are exact; their fp32 sum over d / 32 matrix products a
    digit (at most 6) may truncate at 2^-22 of the largest partial sum each time, which reach bounds within the digits'
    own overlap of 2^-3; the query's digits end at 2^-21 of the row's largest element."""
    return (d / 8 + 5) * 2.0 ** -22 * reach + 2.0 ** -21 * floor


def tolerance(dz, vmax, out_bf16, ref, prior=False):
    """How far an output may be from the 64-bit one.

    With ln 2 < 1, dz (logit_error) bounds the relative error of each weight; base-2 exponential, scales and fp32 sums
    add less than 2^-19.  A weighted mean of values moves by at most twice the weights' relative error times vmax, the
    largest |value|.  The weights' digits enter only the sum of values: int8 ends at half of 2^-21 (fp32 outputs) or
    2^-14 (bf16) of the largest weight of 32 keys, so a tile is off by at most 32 2^-22 (2^-15) of a weight that the
    normaliser holds, 2^-17 (2^-10) vmax together; e4m3's digits are below that (2^-22 or 2^-12 relative, 32 2^-30 or
    32 2^-18 of the largest).  bf16 outputs round at 2^-8.  prior: the scoring pass sums the gists' values with
    weights of two bf16 terms, 2^-16."""
    rel = dz + 2.0 ** -19 + (2.0 ** -16 if prior else 0.0)
    if not out_bf16:
        return 2 * rel * vmax + 2.0 ** -17 * vmax
    return 2 * rel * vmax + 2.0 ** -10 * vmax + 2.0 ** -8 * ref.abs()


def lse_tolerance(dz, lse):
    """The logits' error, and the rounding of ln and of the result."""
    return dz + 2.0 ** -19 + 2.0 ** -21 * abs(lse)
