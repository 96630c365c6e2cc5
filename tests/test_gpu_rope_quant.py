"""Rotary positions and quantised history pages on the GPU, against plain forms in 64 bits.

Tolerances count roundings: HALF_STEP of an output's type (finfo.eps / 2 of the value), ROPE_ERR for a rotation in fp32,
the fp32 sums' terms x 2^-24."""
import math

import numpy as np
import pytest
import torch

from quant_testlib import HALF_STEP, QMAX, ROPE_ERR, Pages, attention64, encode, rope64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import hybrid_sparse_attention_hkv_b200 as hsa

CU = "cuda"


def gen(seed):
    return torch.Generator(CU).manual_seed(seed)


def rand(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=gen(seed), device=CU).to(dtype)


def workspace(n=256):
    return torch.zeros(n, dtype=torch.uint8, device=CU)


def make_rope(rot, axes, layout, mscale=1.0):
    pairs = [rot // 2] if axes == 1 else [rot // 2 - 2 * (rot // 6), rot // 6, rot // 6]
    inv = torch.cat([hsa.rope_freqs(2 * n)[0] for n in pairs]).cuda()
    return hsa.make_rope(inv, layout, pairs, mscale), inv, pairs


def positions(axes, T, seed, far=100000):
    return torch.randint(-far, far, (axes, T), generator=gen(seed), device=CU, dtype=torch.int32)


def within(got, want, bound, what=""):
    got, want = got.double().cpu(), want.double().cpu()
    over = ((got - want).abs() - bound).max().item() if got.numel() else 0.0
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and not over > 0, f"{what}: {over:.3e} over the bound"


# ------------------------------------------------------------------ rotary positions

ROPES = [(64, 64, 1, 0), (64, 64, 3, 1), (64, 16, 1, 1), (64, 48, 3, 0), (128, 128, 3, 0), (128, 128, 1, 1), (128, 96, 3, 1),
         (128, 32, 1, 0), (128, 112, 3, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("d,rot,axes,layout", ROPES)
@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 0), (1, 40, 8), (3, 2, 2), (131, 5, 1)])
def test_rope_and_its_gradient(d, rot, axes, layout, T, Hq, Hk, dtype):
    rope, inv, pairs = make_rope(rot, axes, layout, 1.25)
    pos = positions(axes, T, 1)
    q = rand(T, Hq, d, seed=2, dtype=dtype)
    k = rand(T, Hk, d, seed=3, dtype=dtype) if Hk else None
    for call, sign in ((hsa.hsa_rope, 1.0), (hsa.hsa_rope_bwd, -1.0)):
        qo, ko = torch.empty_like(q), None if k is None else torch.empty_like(k)
        call(rope, pos, q, qo, k, ko)
        for x, y in ((q, qo), (k, ko)):
            if x is not None:
                want, err = rope64(x, pos, inv, pairs, layout, 1.25, sign)
                within(y, want, err + HALF_STEP[dtype] * (want.abs() + err), f"sign {sign}")
                assert torch.equal(y[..., rot:], x[..., rot:])


def test_rope_gradient_against_differences():
    """The rotation is linear, so a difference with any step is its derivative: every entry of dL/dx for L = <g, y>."""
    d, rot, T = 64, 48, 2
    rope, inv, pairs = make_rope(rot, 1, 1, 0.75)
    pos = positions(1, T, 5, 50)
    x, g = rand(T, 1, d, seed=6), rand(T, 1, d, seed=7)
    dx = torch.empty_like(x)
    hsa.hsa_rope_bwd(rope, pos, g, dx)
    steps = torch.zeros(T * d, T, 1, d, device=CU)
    steps.view(T * d, T * d).fill_diagonal_(1.0)
    num = torch.empty(T * d, dtype=torch.float64)
    for i in range(T * d):
        y = torch.empty_like(x)
        hsa.hsa_rope(rope, pos, steps[i], y)
        num[i] = (y.double() * g.double()).sum()
    # both sides err by ROPE_ERR on two products of |g|
    within(dx.flatten(), num, 4 * ROPE_ERR * float(g.abs().max()))


def test_rope_strided_in_place_and_broadcast_rows():
    d, T, Hq, Hk = 128, 37, 6, 2
    rope, inv, pairs = make_rope(128, 3, 0)
    pos = positions(3, T, 8)
    fused = rand(T, Hq + 2 * Hk, d, seed=9, dtype=torch.bfloat16)
    before = fused.clone()
    q, k = fused[:, :Hq], fused[:, Hq:Hq + Hk]
    hsa.hsa_rope(rope, pos, q, q, k, k)  # in place, inside a fused projection
    want, err = rope64(before[:, :Hq + Hk], pos, inv, pairs, 0)
    within(fused[:, :Hq + Hk], want, err + HALF_STEP[torch.bfloat16] * (want.abs() + err))
    assert torch.equal(fused[:, Hq + Hk:], before[:, Hq + Hk:])
    one = rand(1, Hk, d, seed=10, dtype=torch.float16)
    heads_first = torch.zeros(Hk, T, d, dtype=torch.float16, device=CU)
    hsa.hsa_rope(rope, pos, one.expand(T, Hk, d), heads_first.transpose(0, 1))  # one row at every position, [H, T, d] out
    want, err = rope64(one.expand(T, Hk, d), pos, inv, pairs, 0)
    within(heads_first.transpose(0, 1), want, err + HALF_STEP[torch.float16] * (want.abs() + err))


def test_rope_far_positions():
    """The whole int32 range.  The angle in turns is rounded twice in fp64 (2^-53 each) at up to 2^31 / (2 pi) turns:
    an error below 2^31 * 2^-52 = 2^-21 radians on top of ROPE_ERR."""
    d = 128
    rope, inv, pairs = make_rope(d, 1, 0)
    at = torch.tensor([0, 1, -1, 2 ** 20, 2 ** 24 + 1, 2 ** 30, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=CU)
    x = rand(len(at), 3, d, seed=11)
    y = torch.empty_like(x)
    hsa.hsa_rope(rope, at, x, y)
    want, err = rope64(x, at, inv, pairs, 0)
    within(y, want, 3 * err + HALF_STEP[torch.float32] * want.abs())


def test_rope_no_tokens_and_not_finite_values():
    rope, inv, pairs = make_rope(64, 1, 1)
    empty = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=CU)
    hsa.hsa_rope(rope, torch.empty(1, 0, dtype=torch.int32, device=CU), empty, empty.clone())
    part, _, _ = make_rope(32, 1, 1)
    x = torch.ones(1, 2, 64, device=CU)
    x[0, 0, 40], x[0, 0, 41] = float("nan"), float("inf")  # behind the rotated columns: copied, nothing else touched
    y = torch.empty_like(x)
    hsa.hsa_rope(part, torch.tensor([3], dtype=torch.int32, device=CU), x, y)
    assert torch.isnan(y[0, 0, 40]) and torch.isinf(y[0, 0, 41]) and torch.isfinite(y).sum() == 126


# ------------------------------------------------------------------ writing pages

def check_written(pages, lo, hi, codes, scales):
    """Rows [lo, hi) of the pages hold these codes and scales bit for bit; every other byte is as it was (0xAB)."""
    c, s = pages.codes().flatten(0, 1), pages.scales().flatten(0, 1)
    assert torch.equal(c[lo:hi].nan_to_num(-999.0), codes.cpu().nan_to_num(-999.0))
    assert torch.equal(s[lo:hi].nan_to_num(-1.0), scales.cpu().nan_to_num(-1.0))
    raw = pages.raw.cpu()
    row_c, row_s = pages.code_bytes // pages.P, pages.scale_bytes // pages.P
    touched = torch.zeros_like(raw, dtype=torch.bool)
    for g in range(lo, hi):
        p, r = divmod(g, pages.P)
        touched[p, r * row_c:(r + 1) * row_c] = True
        touched[p, pages.off + r * row_s:pages.off + (r + 1) * row_s] = True
    assert (raw[~touched] == 0xAB).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("T,first,P,NP,H", [(1, 0, 1, 1, 1), (1, 6, 7, 2, 40), (23, 5, 7, 4, 3)])
def test_rows_are_quantised_bit_for_bit(T, first, P, NP, H, d, group, fmt, dtype):
    q = hsa.make_quant(fmt, group)
    K, V = rand(T, H, d, seed=20, dtype=dtype), rand(T, H, d, seed=21, dtype=dtype) * 3
    pk, pv = Pages(hsa, q, NP, P, H, d), Pages(hsa, q, NP, P, H, d)
    ws = workspace()
    hsa.hkv_quant_rows(q, K, V, pk.table, pv.table, P, first, ws)
    for x, p in ((K, pk), (V, pv)):
        check_written(p, first, first + T, *encode(x.float().cpu(), fmt, group))
    assert hsa.hsa_status_read(ws) == 0


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_rows_edge_values(fmt):
    """Zeros, the smallest and largest magnitudes, equal magnitudes, signed zeros, infinities and NaN."""
    d, group, H = 64, 32, 2
    q = hsa.make_quant(fmt, group)
    x = rand(9, H, d, seed=22)
    x[0] = 0
    x[1] = -0.0
    x[2] *= 2.0 ** -101 / x[2].abs().max()
    x[3, 0] = 2.0 ** -100
    x[3, 1] *= 3.3e38 / x[3, 1].abs().max()
    x[4] = x[4].sign() * 5.0
    x[5, 0, 3], x[5, 1, 40] = float("nan"), float("inf")
    x[6, 0, 0] = float("-inf")
    x[7, 0] = 1e-42  # subnormal
    x[8, :, 1:] *= 1e-6
    pk, pv = Pages(hsa, q, 1, 9, H, d), Pages(hsa, q, 1, 9, H, d)
    hsa.hkv_quant_rows(q, x, x, pk.table, pv.table, 9, 0, workspace())
    codes, scales = encode(x.cpu(), fmt, group)
    check_written(pk, 0, 9, codes, scales)
    check_written(pv, 0, 9, codes, scales)
    assert torch.isnan(scales).sum() == 3 and scales[0].abs().sum() == 0 and scales[2].abs().sum() == 0


@pytest.mark.parametrize("d,rot,axes,layout", ROPES)
@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_rows_with_rotated_keys(d, rot, axes, layout, fmt):
    """Keys are rotated before they are quantised: every value read back is within half a step of the format of the
    rotated key (plus the rotation's fp32 error and three roundings of scale, quotient and product), values as they come."""
    T, H, P = 13, 3, 16
    for group in (g for g in (32, 64, 128) if g <= d):
        q = hsa.make_quant(fmt, group)
        rope, inv, pairs = make_rope(rot, axes, layout, 1.5)
        pos = positions(axes, T, 23)
        K, V = rand(T, H, d, seed=24, dtype=torch.bfloat16), rand(T, H, d, seed=25, dtype=torch.bfloat16)
        pk, pv = Pages(hsa, q, 1, P, H, d), Pages(hsa, q, 1, P, H, d)
        hsa.hkv_quant_rows(q, K, V, pk.table, pv.table, P, 2, workspace(), rope=rope, pos=pos)
        check_written(pv, 2, 2 + T, *encode(V.float().cpu(), fmt, group))
        want, err = rope64(K, pos, inv, pairs, layout, 1.5)
        amax = want.unflatten(-1, (-1, group)).abs().amax(-1).repeat_interleave(group, -1)
        scale = amax / QMAX[fmt]
        step = torch.maximum(want.abs() * 2.0 ** -4, scale * 2.0 ** -10) if fmt == 0 else scale * 0.5
        within(pk.rows64()[0, 2:2 + T], want, step * (1 + 2.0 ** -16) + 3 * err.amax() + amax * 2.0 ** -20, f"group {group}")


def test_rows_position_from_the_device_and_rows_outside():
    d, group, H, P, NP, T = 64, 64, 2, 4, 3, 5
    q = hsa.make_quant(1, group)
    K, V = rand(T, H, d, seed=26), rand(T, H, d, seed=27)
    codes, scales = encode(K.cpu(), 1, group)
    for host, dev, lo in ((3, 0, 3), (0, 6, 6), (-2, 5, 3), (0, 9, 9), (0, -3, -3), (0, 2 ** 62, None), (0, -2 ** 63, None)):
        pk, pv, ws = Pages(hsa, q, NP, P, H, d), Pages(hsa, q, NP, P, H, d), workspace()
        hsa.hkv_quant_rows(q, K, V, pk.table, pv.table, P, host, ws, first_row_dev=torch.tensor([dev], device=CU))
        if lo is None:
            check_written(pk, 0, 0, codes[:0], scales[:0])
        else:
            a, b = max(lo, 0), min(lo + T, NP * P)
            check_written(pk, a, b, codes[a - lo:b - lo], scales[a - lo:b - lo])
        assert hsa.hsa_status_read(ws) == (0 if lo is not None and 0 <= lo <= NP * P - T else 6)
    # a page without an address is skipped, its neighbours are written
    pk, pv, ws = Pages(hsa, q, NP, P, H, d), Pages(hsa, q, NP, P, H, d), workspace()
    pv.table[1] = 0
    hsa.hkv_quant_rows(q, K, V, pk.table, pv.table, P, 3, ws)
    check_written(pk, 3, 4, codes[:1], scales[:1])
    assert hsa.hsa_status_read(ws) == 6


# ------------------------------------------------------------------ reading pages

def filled(q, NP, P, H, d, seed, spread=1.0):
    p = Pages(hsa, q, NP, P, H, d)
    x = torch.randn(NP, P, H, d, generator=torch.Generator().manual_seed(seed)) * spread
    p.set(*encode(x, q.format, q.group))
    return p


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("P,NP,sel,H", [(1, 1, [0], 1), (37, 5, [0, 2, 4], 3), (200, 3, [1, 1, 0], 12), (128, 2, [1], 130)])
@pytest.mark.parametrize("means", [False, True])
def test_pages_read_back(P, NP, sel, H, d, group, fmt, means):
    q = hsa.make_quant(fmt, group)
    pk, pv = filled(q, NP, P, H, d, 30), filled(q, NP, P, H, d, 31)
    n = len(sel) * P
    Kc, Vc = (torch.empty(n, H, d, dtype=torch.bfloat16, device=CU) for _ in range(2))
    kb = torch.full((-(-n // 128), H, d), -7.0, device=CU) if means else None
    ws = workspace()
    hsa.hkv_gather_quant(q, pk.table, pv.table, torch.tensor(sel, dtype=torch.int32, device=CU), len(sel), P, H, d, Kc, Vc, ws,
                         kbar128=kb)
    k, v = pk.rows64()[sel].flatten(0, 1), pv.rows64()[sel].flatten(0, 1)
    # code * scale is one fp32 product, rounded once more: bit-equal to the same two roundings
    assert torch.equal(Kc.cpu(), k.float().bfloat16()) and torch.equal(Vc.cpu(), v.float().bfloat16())
    if means:
        check_means(kb, k, torch.zeros_like(k))
    assert hsa.hsa_status_read(ws) == 0


def check_means(kb, k, err):
    """128 rows added in fp32: each of 127 sums rounds at 2^-24 of a partial sum of at most sum |k|, and each term has its
    own error (one product, or the rotation's)."""
    for j, rows in enumerate(k.split(128)):
        mag = rows.abs().sum(0)
        bound = (mag * 130 * 2.0 ** -24 + err.split(128)[j].sum(0)) / len(rows)
        within(kb[j], rows.mean(0), bound + 2.0 ** -24 * rows.mean(0).abs(), f"block {j}")


@pytest.mark.parametrize("d,rot,axes,layout", ROPES)
@pytest.mark.parametrize("fmt", [0, 2])
def test_pages_read_back_with_rotated_keys(d, rot, axes, layout, fmt):
    group, H, P, NP, sel = 32, 5, 75, 4, [0, 3]
    q = hsa.make_quant(fmt, group)
    rope, inv, pairs = make_rope(rot, axes, layout, 0.5)
    pk, pv = filled(q, NP, P, H, d, 32), filled(q, NP, P, H, d, 33)
    n = len(sel) * P
    pos = positions(axes, n, 34)
    k, v = pk.rows64()[sel].flatten(0, 1), pv.rows64()[sel].flatten(0, 1)
    want, err = rope64(k, pos, inv, pairs, layout, 0.5)
    err = err + 2.0 ** -23 * k.abs().amax()  # code * scale rounds once before
    for means in (False, True):
        Kc, Vc = (torch.empty(n, H, d, dtype=torch.bfloat16, device=CU) for _ in range(2))
        kb = torch.empty(2, H, d, device=CU) if means else None
        hsa.hkv_gather_quant(q, pk.table, pv.table, torch.tensor(sel, dtype=torch.int32, device=CU), len(sel), P, H, d, Kc, Vc,
                             workspace(), kbar128=kb, rope=rope, pos=pos)
        within(Kc, want, err + HALF_STEP[torch.bfloat16] * (want.abs() + err))
        assert torch.equal(Vc.cpu(), v.float().bfloat16())
        if means:
            check_means(kb, want, err)


def test_bad_pages_are_skipped_by_the_read():
    q, H, d, P = hsa.make_quant(0, 64), 2, 64, 50
    pk, pv = filled(q, 3, P, H, d, 35), filled(q, 3, P, H, d, 36)
    k, v = pk.rows64(), pv.rows64()
    for sel, break_table in (([0, -1, 2], False), ([0, 7, 2], False), ([0, 1, 2], True)):
        tk, tv = pk.table.clone(), pv.table.clone()
        if break_table:
            tk[1], tv[1] = 0, tv[1] + 8
        Kc, Vc = (torch.full((3 * P, H, d), 9.0, dtype=torch.bfloat16, device=CU) for _ in range(2))
        kb, ws = torch.empty(2, H, d, device=CU), workspace()
        hsa.hkv_gather_quant(q, tk, tv, torch.tensor(sel, dtype=torch.int32, device=CU), 3, P, H, d, Kc, Vc, ws, kbar128=kb)
        assert hsa.hsa_status_read(ws) == 6
        zero = torch.zeros_like(k[0])
        for out, x in ((Kc, k), (Vc, v)):
            assert torch.equal(out[:P].cpu(), x[0].float().bfloat16()) and torch.equal(out[2 * P:].cpu(), x[2].float().bfloat16())
            assert (out[P:2 * P] == 9.0).all()
        check_means(kb, torch.cat([k[0], zero, k[2]]), torch.zeros(3 * P, H, d))


# ------------------------------------------------------------------ attention over pages

def attend(q, Q, pk, pv, sel, out_dtype=torch.float32, n_rows=None, scale=0.0, lse=True, ws=None, out=None):
    T, Hq, d = Q.shape
    out = torch.full((T, Hq, d), 5.0, dtype=out_dtype, device=CU) if out is None else out
    ls = torch.full((T, Hq), 5.0, device=CU) if lse else None
    if ws is None:
        ws = workspace(hsa.hkv_attn_quant_workspace_size(T, Hq, pk.H, d, len(sel), pk.P))
    hsa.hkv_attn_quant(q, Q, pk.table, pv.table, torch.tensor(sel, dtype=torch.int32, device=CU), len(sel), pk.P, pk.H, out, ls, ws,
                       n_rows=None if n_rows is None else torch.tensor([n_rows], dtype=torch.int32, device=CU), scale=scale)
    return out, ls, hsa.hsa_status_read(ws)


def check_attention(out, ls, Q, k, v, scale):
    """Scores: d products and their sums in fp32 (taken as 2^-22 a term, the tensor core's adder rounds coarser than
    2^-24), scaled by three more roundings: an absolute error e of the exponent, so weights are off by e relative (both in
    the numerator and in the sum).  Weights add 2^-21 each for exp2, the scales and the split halves; the sums over the rows
    another 2^-21 of sum p |v| <= max |v|."""
    want, lse, mag = attention64(Q.double().cpu(), k, v, scale)
    e = mag * 2.0 ** -21 + 2.0 ** -22
    big = v.abs().amax().item() if v.numel() else 0.0
    within(out, want, (2 * e + 2.0 ** -19) * big + (HALF_STEP[torch.bfloat16] if out.dtype == torch.bfloat16 else 2.0 ** -24) *
           want.abs(), "out")
    if ls is not None:
        within(ls, lse, e + 2.0 ** -20 + 2.0 ** -22 * lse.abs(), "lse")


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("T,g,H,P,NP,sel,n", [
    (1, 1, 1, 1, 1, [0], None), (1, 1, 3, 16, 2, [1], 16), (1, 1, 2, 37, 4, [0, 3], 38), (7, 1, 2, 17, 3, [2, 1, 0], 50),
    (2, 5, 2, 200, 3, [0, 1], 399), (16, 1, 1, 640, 4, [0, 1, 2, 3], None), (9, 2, 3, 33, 2, [0, 1], 65)])
def test_attention_over_pages(T, g, H, P, NP, sel, n, d, group, fmt):
    q = hsa.make_quant(fmt, group)
    pk, pv = filled(q, NP, P, H, d, 40), filled(q, NP, P, H, d, 41)
    Q = rand(T, H * g, d, seed=42, dtype=torch.bfloat16)
    rows = len(sel) * P if n is None else n
    k, v = (p.rows64()[sel].flatten(0, 1)[:rows] for p in (pk, pv))
    for dt in (torch.float32, torch.bfloat16):
        out, ls, st = attend(q, Q, pk, pv, sel, dt, n)
        assert st == 0
        check_attention(out, ls, Q, k, v, 1 / math.sqrt(d))
    out2, ls2, _ = attend(q, Q, pk, pv, sel, torch.bfloat16, n)
    assert torch.equal(out, out2) and torch.equal(ls, ls2)  # deterministic
    out3, _, _ = attend(q, Q, pk, pv, sel, torch.bfloat16, n, lse=False)
    assert torch.equal(out, out3)


@pytest.mark.parametrize("n", [-5, 0, 1, 15, 16, 17, 36, 37, 38, 110, 111, 10 ** 6])
def test_attention_lengths(n):
    """Lengths of zero and one, ends inside a tile and at a page's end, and more than there are; rows behind the end hold
    NaN codes and scales."""
    q, H, d, P, sel = hsa.make_quant(0, 64), 2, 64, 37, [2, 0, 1]
    pk, pv = filled(q, 3, P, H, d, 43), filled(q, 3, P, H, d, 44)
    m = min(max(n, 0), 111)
    k, v = (p.rows64()[sel].flatten(0, 1)[:m] for p in (pk, pv))
    for p in (pk, pv):
        for r in range(m, 111):
            page, row = sel[r // P], r % P
            p.raw[page, row * H * d:(row + 1) * H * d] = 0x7F
            p.raw[page, p.off + row * H * 4:p.off + (row + 1) * H * 4] = 0xFF
    Q = rand(3, 4, d, seed=45, dtype=torch.bfloat16)
    out, ls, st = attend(q, Q, pk, pv, sel, n_rows=n)
    assert st == 0
    if m == 0:
        assert (out == 0).all() and (ls == -math.inf).all()
    else:
        check_attention(out, ls, Q, k, v, 1 / math.sqrt(d))


def test_attention_over_many_splits_joins_them():
    """Enough rows that every split has work, T x heads that fill several query tiles, and a scale of its own."""
    q, H, d, P = hsa.make_quant(1, 128), 2, 128, 3001
    pk, pv = filled(q, 2, P, H, d, 46), filled(q, 2, P, H, d, 47)
    Q = rand(64, 2 * H, d, seed=48, dtype=torch.bfloat16)
    k, v = (p.rows64().flatten(0, 1)[:5555] for p in (pk, pv))
    out, ls, st = attend(q, Q, pk, pv, [0, 1], n_rows=5555, scale=0.25)
    assert st == 0
    check_attention(out, ls, Q, k, v, 0.25)
    # disjoint rows merge by their lse to the whole
    a, la, _ = attend(q, Q, pk, pv, [0], scale=0.25)
    b, lb, _ = attend(q, Q, pk, pv, [1], n_rows=5555 - P, scale=0.25)
    whole = torch.logaddexp(la, lb)
    merged = a * (la - whole).exp()[..., None] + b * (lb - whole).exp()[..., None]
    check_attention(merged, whole, Q, k, v, 0.25)


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_attention_value_scales_over_a_wide_range(fmt):
    """Value scales from 2^-90 to 2^90, rising and falling along the rows, and zero groups: the running reference power of
    two is raised, and small values keep their accuracy where nothing larger drowns them."""
    q, H, d, P = hsa.make_quant(fmt, 32), 1, 64, 96
    pk, pv = filled(q, 2, P, H, d, 49), filled(q, 2, P, H, d, 50)
    codes, scales = pv.codes(), pv.scales()
    for powers in ([-90, 90], [90, -90], [-90, -90], [60, 60]):
        s = scales.clone()
        s[0], s[1] = s[0] * 2.0 ** powers[0], s[1] * 2.0 ** powers[1]
        s[:, ::7, :, 1] = 0
        pv.set(codes, s)
        Q = rand(2, H, d, seed=51, dtype=torch.bfloat16)
        k, v = (p.rows64().flatten(0, 1) for p in (pk, pv))
        out, ls, _ = attend(q, Q, pk, pv, [0, 1])
        check_attention(out, ls, Q, k, v, 1 / math.sqrt(d))


def test_attention_query_magnitudes():
    """Queries of very different and of extreme magnitudes (scores that saturate the softmax), and all-zero queries."""
    q, H, d, P = hsa.make_quant(0, 64), 1, 64, 150
    pk, pv = filled(q, 1, P, H, d, 52), filled(q, 1, P, H, d, 53)
    Q = rand(6, H, d, seed=54, dtype=torch.bfloat16)
    Q[0] = 0
    Q[1] *= 1e-30
    Q[2, :, ::2] *= 1e-7
    Q[3] *= 8
    k, v = pk.rows64()[0], pv.rows64()[0]
    out, ls, _ = attend(q, Q, pk, pv, [0])
    for i in range(6):
        check_attention(out[i:i + 1], ls[i:i + 1], Q[i:i + 1], k, v, 1 / 8)
    big = rand(1, H, d, seed=55, dtype=torch.bfloat16) * 1e30  # one row takes all the weight
    out, ls, _ = attend(q, big, pk, pv, [0])
    top = int((k[:, 0] @ big[0, 0].double().cpu()).argmax())
    within(out[0, 0], v[top, 0], 2.0 ** -20 * v.abs().max())


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("T,g,H,P,sel,n", [(1, 1, 4, 33, [1, 1, 0], 70), (3, 4, 8, 95, [2, 0, 2], None), (9, 1, 6, 64, [0, 0], 127),
                                           (64, 1, 4, 5, [2, 2, 2], 14)])
def test_attention_of_neighbouring_heads_and_pages_selected_twice(T, g, H, P, sel, n, d, group, fmt):
    q = hsa.make_quant(fmt, group)
    pk, pv = filled(q, 3, P, H, d, 140), filled(q, 3, P, H, d, 141)
    Q = rand(T, H * g, d, seed=142, dtype=torch.bfloat16)
    rows = len(sel) * P if n is None else n
    k, v = (p.rows64()[sel].flatten(0, 1)[:rows] for p in (pk, pv))
    out, ls, st = attend(q, Q, pk, pv, sel, n_rows=n)
    assert st == 0
    check_attention(out, ls, Q, k, v, 1 / math.sqrt(d))


@pytest.mark.parametrize("T", [5, 12])
def test_attention_scales_below_the_exponent_range(T):
    """Zero and tiny queries with scales whose product with them is below fp32's range: the rows' plain mean, also where a
    tile's last rows are masked."""
    q, H, d, P = hsa.make_quant(0, 64), 2, 64, 150
    pk, pv = filled(q, 2, P, H, d, 152), filled(q, 2, P, H, d, 153)
    n = 2 * P - 7
    k, v = (p.rows64().flatten(0, 1)[:n] for p in (pk, pv))
    Q = rand(T, H, d, seed=154, dtype=torch.bfloat16)
    Q[0] = 0
    Q[1] *= 1e-36
    for scale in (1e-9, 1e-20, 1e-38):
        out, ls, st = attend(q, Q, pk, pv, [0, 1], n_rows=n, scale=scale)
        assert st == 0
        check_attention(out, ls, Q, k, v, torch.tensor(scale).item())


def test_attention_not_finite_groups_reach_their_own_head_only():
    q, H, d, P = hsa.make_quant(0, 64), 3, 64, 40
    for which in ("k", "v"):
        pk, pv = filled(q, 1, P, H, d, 56), filled(q, 1, P, H, d, 57)
        Q = rand(2, H, d, seed=58, dtype=torch.bfloat16)
        clean, _, _ = attend(q, Q, pk, pv, [0])
        p = pk if which == "k" else pv
        s = p.scales()
        s[0, 17, 1] = float("nan")
        p.set(p.codes(), s)
        out, ls, _ = attend(q, Q, pk, pv, [0])
        assert torch.isnan(out[:, 1]).all()
        assert torch.equal(out[:, [0, 2]], clean[:, [0, 2]])
        assert torch.isnan(ls[:, 1]).all() == (which == "k") and torch.isfinite(ls[:, [0, 2]]).all()


def test_attention_bad_pages_are_not_attended_to():
    q, H, d, P = hsa.make_quant(2, 32), 2, 128, 45
    pk, pv = filled(q, 3, P, H, d, 59), filled(q, 3, P, H, d, 60)
    Q = rand(2, H, d, seed=61, dtype=torch.bfloat16)
    k, v = (p.rows64()[[0, 2]].flatten(0, 1) for p in (pk, pv))
    for sel, broken in (([0, -1, 2], False), ([0, 3, 2], False), ([0, 1, 2], True)):
        keep = pv.table.clone()
        if broken:
            pv.table[1] = 0
        out, ls, st = attend(q, Q, pk, pv, sel)
        assert st == 6
        check_attention(out, ls, Q, k, v, 1 / math.sqrt(d))
        pv.table.copy_(keep)
    out, ls, st = attend(q, Q, pk, pv, [-1, 5, 9][:3])
    assert st == 6 and (out == 0).all() and (ls == -math.inf).all()


# ------------------------------------------------------------------ streams, graphs, calls together

def test_another_stream_and_captured_graph_of_a_decode_step():
    """A step that appends one token at a position held on the device, then attends to all rows so far: captured once,
    replayed with new inputs and positions, on a stream of its own."""
    q, H, d, P, NP = hsa.make_quant(0, 128), 4, 128, 20, 3
    rope, inv, pairs = make_rope(128, 1, 1)
    steps = 45
    Ks, Vs, Qs = (rand(steps, H, d, seed=70 + i, dtype=torch.bfloat16) for i in range(3))
    pk, pv = Pages(hsa, q, NP, P, H, d), Pages(hsa, q, NP, P, H, d)
    k, v, x, xr = (torch.zeros(1, H, d, dtype=torch.bfloat16, device=CU) for _ in range(4))
    pos, row, n = (torch.zeros(1, dtype=dt, device=CU) for dt in (torch.int32, torch.int64, torch.int32))
    sel = torch.arange(NP, dtype=torch.int32, device=CU)
    out, ls = torch.empty(1, H, d, device=CU), torch.empty(1, H, device=CU)
    ws = workspace(hsa.hkv_attn_quant_workspace_size(1, H, H, d, NP, P))

    def step():
        hsa.hkv_quant_rows(q, k, v, pk.table, pv.table, P, 0, ws, first_row_dev=row, rope=rope, pos=pos)
        hsa.hsa_rope(rope, pos, x, xr)
        hsa.hkv_attn_quant(q, xr, pk.table, pv.table, sel, NP, P, H, out, ls, ws, n_rows=n)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    eager, captured = [], []
    for mode, got in ((0, eager), (1, captured)):
        pk.raw.fill_(0xAB)
        pv.raw.fill_(0xAB)
        for i in range(steps):
            k.copy_(Ks[i:i + 1]), v.copy_(Vs[i:i + 1]), x.copy_(Qs[i:i + 1])
            pos.fill_(i), row.fill_(i), n.fill_(i + 1)
            graph.replay() if mode else step()
            got.append((out.clone(), ls.clone(), xr.clone()))
    assert hsa.hsa_status_read(ws) == 0
    for a, b in zip(eager, captured):
        assert all(torch.equal(s, t) for s, t in zip(a, b))
    kk, vv = pk.rows64().flatten(0, 1), pv.rows64().flatten(0, 1)
    for i in (0, 19, 20, 44):
        check_attention(captured[i][0], captured[i][1], captured[i][2], kk[:i + 1], vv[:i + 1], 1 / math.sqrt(d))


def test_two_streams_at_once():
    """Two calls in flight on two streams, each with a workspace of its own, give what they give one after the other."""
    q, H, d, P = hsa.make_quant(1, 64), 4, 64, 3000
    pk, pv = filled(q, 2, P, H, d, 90), filled(q, 2, P, H, d, 91)
    Qs = [rand(9, H, d, seed=92 + i, dtype=torch.bfloat16) for i in range(2)]
    want = [attend(q, x, pk, pv, [0, 1]) for x in Qs]
    sel = torch.arange(2, dtype=torch.int32, device=CU)
    streams = [torch.cuda.Stream() for _ in Qs]
    got = []
    torch.cuda.synchronize()
    for s, x in zip(streams, Qs):
        ws = workspace(hsa.hkv_attn_quant_workspace_size(9, H, H, d, 2, P))
        out, ls = torch.empty(9, H, d, device=CU), torch.empty(9, H, device=CU)
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(20):
            hsa.hkv_attn_quant(q, x, pk.table, pv.table, sel, 2, P, H, out, ls, ws, stream=s)
        got.append((out, ls, ws))
    torch.cuda.synchronize()
    for (o, ls, _), (a, b, ws) in zip(want, got):
        assert torch.equal(o, a) and torch.equal(ls, b) and hsa.hsa_status_read(ws) == 0


def test_rows_beyond_two_to_the_31_elements():
    """A page of more than 2^31 code bytes: offsets are 64-bit."""
    q, H, d = hsa.make_quant(0, 128), 40, 128
    P = 430000  # x 5120 = 2.2e9 bytes
    nb, off = hsa.hkv_quant_page_size(q, P, H, d)
    pages = [torch.zeros(nb, dtype=torch.uint8, device=CU) for _ in range(2)]
    tk, tv = (torch.tensor([p.data_ptr()], dtype=torch.int64, device=CU) for p in pages)
    K, V = rand(3, H, d, seed=80, dtype=torch.bfloat16), rand(3, H, d, seed=81, dtype=torch.bfloat16)
    ws = workspace(hsa.hkv_attn_quant_workspace_size(1, H, H, d, 1, P))
    hsa.hkv_quant_rows(q, K, V, tk, tv, P, P - 3, ws)
    for p, x in zip(pages, (K, V)):
        codes, scales = encode(x.float().cpu(), 0, 128)
        at = (P - 3) * H * d
        assert torch.equal(p[at:at + 3 * H * d].cpu().view(torch.float8_e4m3fn).float().view(3, H, d), codes)
        assert torch.equal(p[off + (P - 3) * H * 4:off + P * H * 4].cpu().view(torch.float32).view(3, H, 1), scales)
    # zero rows score 0 and weigh 1 each; the last three answer as themselves
    Q = rand(1, H, d, seed=82, dtype=torch.bfloat16)
    out, ls = torch.empty(1, H, d, device=CU), torch.empty(1, H, device=CU)
    hsa.hkv_attn_quant(q, Q, tk, tv, torch.zeros(1, dtype=torch.int32, device=CU), 1, P, H, out, ls, ws, scale=1.0)
    k, v = ((codes.double().unflatten(-1, (-1, 128)) * s.double()[..., None]).flatten(-2)
            for codes, s in (encode(x.float().cpu(), 0, 128) for x in (K, V)))
    s = torch.einsum("hd,nhd->hn", Q[0].double().cpu(), k)
    total = s.exp().sum(-1) + (P - 3)
    e = s.abs().max().item() * 2.0 ** -20 + 2.0 ** -18
    within(ls[0], total.log(), e + 2.0 ** -22 * total.log())
    want = torch.einsum("hn,nhd->hd", s.exp(), v) / total[:, None]
    weight = torch.einsum("hn,nhd->hd", s.exp(), v.abs()) / total[:, None]
    within(out[0], want, 4 * e * weight + 2.0 ** -24 * v.abs().max())
