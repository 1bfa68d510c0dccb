"""A plain model of the 8-bit cache on the CPU (include/woq_kv8.h), in 64 bits where numbers are
computed and in fp32 where the definition names a rounding.  Shares no code with the library."""
from __future__ import annotations

import numpy as np
import torch

BLOCK = 64


def bf16(x):
    return x.to(torch.bfloat16)


def quantise(x, fmt):
    """x [64, D] bf16 of one block and head -> values [64, D] the block stands for (fp64), codes, scale."""
    x = x.float()
    top = x.abs().max()
    if top == 0:
        return torch.zeros(x.shape, dtype=torch.float64), torch.zeros_like(x), 0.0
    if fmt == 0:
        s = torch.tensor(np.float32(top.item()) / np.float32(127.0))
        c = torch.round(x / s)
    else:
        e = int(np.ceil(np.log2(np.float64(top.item()) / 448.0)))
        s = torch.tensor(np.float32(2.0 ** max(e, -126)))
        c = (x / s).to(torch.float8_e4m3fn).float()
    return c.double() * s.double(), c, float(s)


class Seq:
    """One sequence of one layer: tokens in bf16, [tokens, H, D]."""

    def __init__(self, heads, dim):
        self.k = torch.zeros((0, heads, dim), dtype=torch.bfloat16)
        self.v = torch.zeros((0, heads, dim), dtype=torch.bfloat16)
        self.pk = torch.zeros((0, heads, dim), dtype=torch.bfloat16)
        self.pv = torch.zeros((0, heads, dim), dtype=torch.bfloat16)

    def extend(self, k, v):
        self.k, self.v = torch.cat([self.k, k]), torch.cat([self.v, v])

    def accept(self, mask):
        rows = [j for j in range(8) if mask >> j & 1]
        self.k, self.v = torch.cat([self.k, self.pk[rows]]), torch.cat([self.v, self.pv[rows]])

    def clone(self):
        s = Seq(self.k.shape[1], self.k.shape[2])
        s.k, s.v, s.pk, s.pv = self.k, self.v, self.pk, self.pv
        return s

    def values(self, fmt):
        """fp64 keys and values of the accepted tokens, as the cache stands for them."""
        out = []
        for x in (self.k, self.v):
            y = x.double().clone()
            for b in range(x.shape[0] // BLOCK):
                for h in range(x.shape[1]):
                    y[b * BLOCK:(b + 1) * BLOCK, h] = quantise(x[b * BLOCK:(b + 1) * BLOCK, h], fmt)[0]
            out.append(y)
        return out

    def read(self, fmt, first, count):
        """What woq_kv8_read gives, bf16: the product code * s rounded to fp32, then to bf16."""
        out = []
        for y, p in zip(self.values(fmt), (self.pk, self.pv)):
            out.append(bf16(torch.cat([y.float(), p.float()]))[first:first + count])
        return out


def attention(seq, fmt, q, vis, scale, window=0, sinks=0):
    """q [rows, Hq, D] bf16; vis: a mask for each row.  Returns out [rows, Hq, D] fp64 and a bound on
    the kernel's error per element.

    The bound: weights are rounded to f16 (half a step, 2^-11 relative), those below 2^-14 * 2^-7 of
    the largest by 2^-25 * 2^-7 in all (f16's subnormal step, the factor 2^7 they carry); scores
    are fp32 sums of D exact products (each partial sum off by 2^-24, twice for the running order
    of the tensor core's own sums), two fp32 roundings of factors and one of the difference with the maximum;
    queries below 2^-14 of a row's largest lose 2^-25 of it; ex2 is good to 2^-22; sums over N
    tokens of positive weights lose at most (N / 256 + 300) 2^-24 (a warp adds 8 at a time, lanes, warps and
    CTAs join what they have).  The result is rounded to bf16: half a step, 2^-8 relative."""
    k, v = seq.values(fmt)
    rows, hq, d = q.shape
    h = k.shape[1]
    out = torch.zeros((rows, hq, d), dtype=torch.float64)
    bound = torch.zeros_like(out)
    for m in range(rows):
        seen = [j for j in range(8) if vis[m] >> j & 1]
        kk = torch.cat([k, seq.pk[seen].double()])
        vv = torch.cat([v, seq.pv[seen].double()])
        at = np.arange(len(kk))
        if window:
            at = at[(at < sinks) | (at >= len(kk) - window)]
        if len(at) == 0:
            continue
        kk, vv = kk[at].repeat_interleave(hq // h, 1), vv[at].repeat_interleave(hq // h, 1)
        qq = q[m].double()
        s = torch.einsum("hd,nhd->hn", qq, kk) * scale
        w = torch.softmax(s, -1)
        out[m] = torch.einsum("hn,nhd->hd", w, vv)
        mag = torch.einsum("hd,nhd->hn", qq.abs(), kk.abs()) * abs(scale)  # sum of |products|
        top = qq.abs().amax(-1, keepdim=True) * kk.abs().sum(-1).T * abs(scale) * 2.0 ** -25
        ds = mag * (2 * d + 4) * 2.0 ** -24 + top + (s.abs() + s.abs().amax(-1, keepdim=True)) * 2.0 ** -22
        rel = 2 * ds.amax(-1, keepdim=True) + 2.0 ** -20 + (len(at) / 256 + 300) * 2.0 ** -24
        a = torch.einsum("hn,nhd->hd", w, vv.abs())
        lost = len(at) * 2.0 ** -32 * vv.abs().amax(0)
        err = a * (2.0 ** -11 + 2 * rel) + lost
        bound[m] = err + (out[m].abs() + err) * 2.0 ** -8 + 2.0 ** -130
    return out, bound


def rotate(x, table, pos, axis_of, interleaved=False):
    """x [rows, heads, D] fp32, table [positions, half, 2] fp32: the definition, rounding by rounding."""
    x = x.float()
    half = table.shape[1]
    p = torch.stack([pos[a].long() for a in axis_of], 1)
    cs = table[p, torch.arange(half)]
    c, s = cs[..., 0][:, None], cs[..., 1][:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    return bf16(y)


def tree_masks(widths):
    """Masks of a root and levels of the given widths, only the first choice of each going on."""
    path, rows = 1, [1]
    for w in widths:
        first = len(rows)
        rows += [path | 1 << (first + j) for j in range(w)]
        path |= 1 << first
    return rows
