"""Plain forms, in 64 bits, of rotary positions and of the quantised history pages."""
from __future__ import annotations

import numpy as np
import torch

QMAX = {0: 448.0, 1: 127.0, 2: 7.0}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# Rotating in fp32 (rope.cuh): the reduced angle, at most pi / 4, is rounded three times (its rest, pi / 2, their product:
# 2.5 * 2^-24 of 0.79, below 2^-23), the series of sin and cos rounds within two halves of an ulp (2^-23), cos x mscale, two
# products and a sum round at 2^-24 each: below 2^-21 of |mscale| (|a| + |b|).
ROPE_ERR = 2.0 ** -21


def rope64(x, pos, inv_freq, axis_pairs, layout, mscale=1.0, sign=1.0):
    """x [T, H, d] (any float type), pos int [n_axes, T] -> (float64 rotated rows, bound of the fp32 error)."""
    x = x.double().cpu().numpy()
    pos = np.asarray(pos.cpu().numpy(), dtype=np.longdouble).reshape(len(axis_pairs), -1)
    f = np.asarray(inv_freq.double().cpu().numpy(), dtype=np.longdouble)
    axis = np.repeat(np.arange(len(axis_pairs)), axis_pairs)
    ang = sign * pos[axis].T * f
    cos, sin = np.cos(ang).astype(np.float64)[:, None], np.sin(ang).astype(np.float64)[:, None]
    rot = 2 * len(f)
    ia, ib = (np.arange(rot // 2), np.arange(rot // 2) + rot // 2) if layout == 1 else (np.arange(0, rot, 2),
                                                                                       np.arange(1, rot, 2))
    y, err = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = mscale * (a * cos - b * sin)
    y[..., ib] = mscale * (b * cos + a * sin)
    err[..., ia] = err[..., ib] = ROPE_ERR * abs(mscale) * (np.abs(a) + np.abs(b))
    return torch.from_numpy(y), torch.from_numpy(err)


def encode(x, fmt, group):
    """x float32 [..., d] on the CPU -> (codes as float32 values [..., d], scales float32), in the definition's fp32 steps."""
    q = x.unflatten(-1, (-1, group))
    a = q.abs().amax(-1)
    kept = torch.isfinite(a) & (a >= 2.0 ** -100)
    qmax = torch.tensor(QMAX[fmt])
    scale = torch.where(kept, a * torch.reciprocal(qmax), torch.zeros(()))
    inv = torch.where(kept, torch.reciprocal(a) * qmax, torch.zeros(()))
    finite = torch.isfinite(q).all(-1)
    scale = torch.where(finite, scale, torch.full((), float("nan")))
    v = q * inv[..., None]
    v = v.to(torch.float8_e4m3fn).float() if fmt == 0 else v.round()
    v = torch.where(finite[..., None], v, torch.zeros(()))
    return v.flatten(-2), scale


class Pages:
    """NP quantised pages of K (or V) as one byte tensor, with views of their parts."""

    def __init__(self, hsa, quant, NP, P, H, d, device="cuda", fill=0xAB):
        self.q, self.NP, self.P, self.H, self.d = quant, NP, P, H, d
        self.bytes, self.off = hsa.hkv_quant_page_size(quant, P, H, d)
        self.raw = torch.full((NP, self.bytes), fill, dtype=torch.uint8, device=device)
        self.table = torch.tensor([self.raw[p].data_ptr() for p in range(NP)], dtype=torch.int64, device=device)
        self.code_bytes = P * H * d // (2 if quant.format == 2 else 1)
        self.scale_bytes = 4 * P * H * (d // quant.group)

    def codes(self):
        """float32 values [NP, P, H, d] of the codes (CPU)."""
        c = self.raw[:, :self.code_bytes].contiguous().cpu().unflatten(1, (self.P, self.H, -1))
        if self.q.format == 0:
            return c.view(torch.float8_e4m3fn).float()
        if self.q.format == 1:
            return c.view(torch.int8).float()
        s = c.view(torch.int8)
        return torch.stack([(s << 4) >> 4, s >> 4], -1).flatten(-2).float()

    def scales(self):
        c = self.raw[:, self.off:self.off + self.scale_bytes].contiguous().cpu()
        return c.view(torch.float32).unflatten(1, (self.P, self.H, -1))

    def set(self, codes, scales):
        """Fill from code values and scales ([NP, P, H, ...] float32, CPU)."""
        if self.q.format == 0:
            c = codes.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            c = codes.to(torch.int8).view(torch.uint8)
            if self.q.format == 2:
                c = (c[..., 0::2] & 15) | (c[..., 1::2] << 4)
        self.raw[:, :self.code_bytes] = c.flatten(1).to(self.raw.device)
        s = scales.float().contiguous().flatten(1).view(torch.uint8)
        self.raw[:, self.off:self.off + self.scale_bytes] = s.to(self.raw.device)

    def rows64(self):
        """float64 rows [NP, P, H, d] the pages stand for."""
        return (self.codes().double().unflatten(-1, (-1, self.q.group)) * self.scales().double()[..., None]).flatten(-2)


def attention64(q, k, v, scale):
    """q [T, Hq, d], k / v [n, H, d] float64 -> (out, lse, bound of the fp32 kernel's absolute error in the scores)."""
    T, Hq, d = q.shape
    H = k.shape[1]
    qq = q.unflatten(1, (H, Hq // H))
    s = torch.einsum("thgd,nhd->thgn", qq, k) * scale
    lse = torch.logsumexp(s, -1)
    o = torch.einsum("thgn,nhd->thgd", torch.softmax(s, -1), v)
    mag = torch.einsum("thgd,nhd->thgn", qq.abs(), k.abs()) * scale
    return o.flatten(1, 2), lse.flatten(1, 2), float(mag.max()) if mag.numel() else 0.0
