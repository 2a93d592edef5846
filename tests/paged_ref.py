"""Plain 64-bit forms of the paged-cache operators, for the tests: loops over
sequences and heads, elementary torch operations on whatever device the inputs
are on, and next to each result the bound that its rounding allows.

Half a step of a type is eps / 2 relative to the value: HALF for bf16.
"""
import math

import torch

HALF = 2.0 ** -8      # bf16: one rounding moves a value by at most 2^-8 of itself
FP32 = 2.0 ** -24


def rope(x, weight, positions, freqs, layout, amplitude, eps):
    """(y, bound): x [T, H, d] normed by head (weight [d] or None) and turned; all in fp64."""
    x = x.double()
    d = x.shape[-1]
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    y, near = x.clone(), x.abs()
    if freqs is not None:
        n = freqs.numel()
        t = positions.double()[:, None, None] * freqs
        c, s = torch.cos(t) * amplitude, torch.sin(t) * amplitude
        ia, ib = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        near = near.clone()
        near[..., ia] = near[..., ib] = amplitude * (a.abs() + b.abs())
    # the rounding to bf16; in fp32: the norm (a sum of d squares, a square root and two products, d + 8 roundings of
    # which half the sum's count), the angle (2 pi FP32) and the sine (a few FP32), two products and a sum
    bound = HALF * y.abs() + (d / 2 + 40) * FP32 * near
    return y, bound * (1 + HALF)


def attention(q, k, v, lim, scale):
    """One sequence: q [n, Hq, d], k, v [S, Hk, d], lim [n] keys seen -> (out, lse, bound of out, bound of lse).

    The kernels' roundings: scores in fp32 (d products and sums: at most d FP32 sum |q_c k_c|), each weight to bf16
    before the second product (HALF of it), the sums in fp32, the result to bf16."""
    n, Hq, d = q.shape
    grp = Hq // k.shape[1]
    out = torch.zeros((n, Hq, d), dtype=torch.float64, device=q.device)
    ob = torch.zeros_like(out)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    lb = torch.zeros_like(lse)
    for i in range(n):
        S = int(lim[i])
        if S == 0:
            continue
        for h in range(Hq):
            kk, vv, qq = k[:S, h // grp].double(), v[:S, h // grp].double(), q[i, h].double()
            x = kk @ qq * scale
            ds = float((kk.abs() @ qq.abs()).max()) * scale * (d + 4) * FP32
            z = torch.logsumexp(x, 0)
            p = torch.exp(x - z)
            out[i, h] = p @ vv
            far = p @ vv.abs()
            # a weight over the sum: twice the score's error and two exponentials' (2^-21), and the sums of S terms,
            # whose error is at most S FP32 and in truth its root
            soft = 2 * ds + 2.0 ** -20 + (math.sqrt(S) + 16) * FP32
            ob[i, h] = (HALF * (out[i, h].abs() + far) + soft * far) * (1 + HALF)
            lse[i, h] = z
            lb[i, h] = ds + 2.0 ** -20 + 4 * FP32 * (abs(float(z)) + abs(float(x.max())))
    return out, lse, ob, lb


def close(got, want, bound, what):
    got = got.double()
    bad = ~((got - want).abs() <= bound + 1e-30)
    if bool(bad.any()):
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values out of bounds, first at {at}: got "
                             f"{float(got[tuple(at)])}, want {float(want[tuple(at)])} within {float(bound[tuple(at)])}")


class Cache:
    """A paged cache whose every row that no sequence holds is `fill`; held and new: rows of each sequence."""

    def __init__(self, held, new, H, d, page, seed, fill=float("nan"), device="cuda", extra=3):
        g = torch.Generator().manual_seed(seed)
        self.held, self.new, self.page, self.d, self.H = held, new, page, d, H
        self.lens = [h + n for h, n in zip(held, new)]
        need = [max(1, -(-l // page)) for l in self.lens]
        total = sum(need) + extra
        order = torch.randperm(total, generator=g)
        self.table = torch.full((len(held), max(need) + 1), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n].to(torch.int32)
            at += n
        self.k = [torch.randn((l, H, d), generator=g).to(torch.bfloat16) for l in self.lens]
        self.v = [torch.randn((l, H, d), generator=g).to(torch.bfloat16) for l in self.lens]
        self.kpages = torch.full((total, page, H, d), fill, dtype=torch.bfloat16)
        self.vpages = torch.full((total, page, H, d), fill, dtype=torch.bfloat16)
        for b, l in enumerate(self.lens):
            for r0 in range(0, l, page):
                n = min(page, l - r0)
                pg = int(self.table[b, r0 // page])
                self.kpages[pg, :n] = self.k[b][r0:r0 + n]
                self.vpages[pg, :n] = self.v[b][r0:r0 + n]
        self.seqlens = torch.tensor(self.lens, dtype=torch.int32)
        self.cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32)
        for f in ("table", "kpages", "vpages", "seqlens", "cu"):
            setattr(self, f, getattr(self, f).to(device))
        self.k = [x.to(device) for x in self.k]
        self.v = [x.to(device) for x in self.v]

    @property
    def longest(self):
        return max(1, max(self.lens))
