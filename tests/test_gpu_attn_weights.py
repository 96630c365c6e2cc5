"""Weights of the attention over quantised pages keep their bits whatever stands beside them: rows with large value scales
that nothing attends to, and rows that draw the attention and carry nothing over a long tail."""
import math

import pytest
import torch

from quant_testlib import QMAX, Pages, encode

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import hybrid_sparse_attention_hkv_b200 as hsa

CU = "cuda"


def sums(units):
    """What the sums may be off by, of sum p |v|, where a warp has that many units of 32 rows: 2 x 3 products of each into
    an accumulator, 2^-22 a product (the tensor core's adder rounds coarser than 2^-24).  exp2 is within 2^-22, in the
    weight and in the sum; weight x value scale and the code products round at 2^-24; four warps, then up to 74 + 8 parts
    of the splits, are added in fp32 with weights of 2^-22 each: 2 + 1 + 1 + 22 of 2^-22."""
    return (6 * units + 26) * 2.0 ** -22


def bounded(out, lse, Q, pk, pv, n=None, units=1):
    """Each output against 64 bits, bounded by what it is the sum of: row r weighs p_r, off by its score's error e_r (as in
    the attention's own tests, for the row's own magnitude) and by the mean of those in the sum.

    What a value adds that is itself zero, beside others of its group that are not, is not in that sum.  Weights are scaled,
    by the largest w = p x value scale of 32 rows, to below 2^15 with that one at 2^14 or more; a half then holds 2^-24 or
    its multiples, so what the first half leaves is known to 2^-25 of 2^-12: 2^-51 of the largest w.  Of 32 rows of codes of
    at most qmax that makes 2^-46 x qmax x w, and over all rows at most the sum of that over w_r."""
    T, Hq, d = Q.shape
    scale = 1.0
    k, v = (x.rows64().flatten(0, 1)[:n] for x in (pk, pv))
    most = (pv.scales().double() * QMAX[pv.q.format]).repeat_interleave(pv.q.group, -1).flatten(0, 1)[:n]
    H = k.shape[1]
    q = Q.double().cpu().unflatten(1, (H, Hq // H))
    s = torch.einsum("thgd,nhd->thgn", q, k) * scale
    p = torch.softmax(s, -1)
    e = torch.einsum("thgd,nhd->thgn", q.abs(), k.abs()) * scale * 2.0 ** -21 + 2.0 ** -22
    mean = (p * e).sum(-1)
    want = torch.einsum("thgn,nhd->thgd", p, v).flatten(1, 2)
    mag = torch.einsum("thgn,nhd->thgd", p, v.abs())
    bound = torch.einsum("thgn,nhd->thgd", p * e, v.abs()) + mag * (mean[..., None] + sums(units))
    off = (out.double().cpu() - want).abs()
    bound = bound + 2.0 ** -46 * torch.einsum("thgn,nhd->thgd", p, most)
    bound = bound.flatten(1, 2) + 2.0 ** -24 * want.abs() + 2.0 ** -149
    worst = (off / bound).max().item()
    assert worst <= 1, f"{worst:.3g} times the bound; {(off / mag.flatten(1, 2)).max().item():.3g} of sum p |v|"
    ls = torch.logsumexp(s, -1).flatten(1, 2)
    assert ((lse.double().cpu() - ls).abs() <= mean.flatten(1, 2) + 2.0 ** -20 + 2.0 ** -22 * ls.abs()).all()


def attend(q, Q, pk, pv, n_rows=None, scale=1.0):
    T, Hq, d = Q.shape
    out, lse = torch.full((T, Hq, d), 5.0, device=CU), torch.full((T, Hq), 5.0, device=CU)
    sel = torch.arange(pk.NP, dtype=torch.int32, device=CU)
    ws = torch.zeros(hsa.hkv_attn_quant_workspace_size(T, Hq, pk.H, d, pk.NP, pk.P), dtype=torch.uint8, device=CU)
    n = None if n_rows is None else torch.tensor([n_rows], dtype=torch.int32, device=CU)
    hsa.hkv_attn_quant(q, Q, pk.table, pv.table, sel, pk.NP, pk.P, pk.H, out, lse, ws, n_rows=n, scale=scale)
    assert hsa.hsa_status_read(ws) == 0
    return out, lse


def cache(fmt, group, d, NP, P, H, T, seed):
    """Pages, codes and scales to be changed, and queries that are all near one positive vector, so that the row of codes
    c everywhere scores about c x its scale x the queries' sum."""
    g = torch.Generator().manual_seed(seed)
    q = hsa.make_quant(fmt, group)
    pk, pv = (Pages(hsa, q, NP, P, H, d) for _ in range(2))
    Q = (0.25 + 0.02 * torch.randn(T, H, d, generator=g)).bfloat16()
    ck, sk = encode(0.5 * torch.randn(NP, P, H, d, generator=g), fmt, group)
    cv, sv = encode(torch.randn(NP, P, H, d, generator=g), fmt, group)
    return q, pk, pv, Q.to(CU), ck, sk, cv, sv


def score_row(ck, sk, page, row, Q, value):
    """Row `row` of page `page` scores about `value` (a sign for all its columns)."""
    ck[page, row] = 1.0
    sk[page, row] = value / Q[0].float().cpu().sum(-1)[:, None]


SHAPES = [(64, 32, 1, 1), (64, 64, 3, 9), (128, 128, 4, 1), (128, 64, 2, 12), (128, 32, 1, 3)]


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("d,group,H,T", SHAPES)
@pytest.mark.parametrize("NP,P", [(1, 32), (2, 96), (3, 700)])
@pytest.mark.parametrize("power", [12, 26, 60])
def test_large_values_that_nothing_attends_to(fmt, d, group, H, T, NP, P, power):
    """One row's value scales are 2^power times the others', and its score 80 below theirs: what it adds is 2^-115 of
    its values.  It is the first row, one in the middle or the last."""
    q, pk, pv, Q, ck, sk, cv, sv = cache(fmt, group, d, NP, P, H, T, 200)
    for page, row in ((0, 0), (NP - 1, P // 2), (NP - 1, P - 1)):
        k, ks, vs = ck.clone(), sk.clone(), sv.clone()
        score_row(k, ks, page, row, Q, -80.0)
        vs[page, row] *= 2.0 ** power
        pk.set(k, ks)
        pv.set(cv, vs)
        bounded(*attend(q, Q, pk, pv), Q, pk, pv)


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("d,group,H,T", SHAPES)
@pytest.mark.parametrize("NP,P", [(1, 32), (1, 128), (4, 1000)])
@pytest.mark.parametrize("nats", [9, 14, 18, 30])
@pytest.mark.parametrize("outlier", [False, True])
def test_a_row_that_draws_the_attention_over_a_long_tail(fmt, d, group, H, T, NP, P, nats, outlier):
    """The first row scores `nats` above the others and has values of zero, or of zero but for one column of each group:
    the other columns are what the tail adds up to."""
    q, pk, pv, Q, ck, sk, cv, sv = cache(fmt, group, d, NP, P, H, T, 201)
    score_row(ck, sk, 0, 0, Q, float(nats))
    cv[0, 0] = 0.0
    if outlier:
        cv[0, 0].unflatten(-1, (-1, group))[..., 5] = 7.0
    else:
        sv[0, 0] = 0.0
    pk.set(ck, sk)
    pv.set(cv.abs(), sv)
    bounded(*attend(q, Q, pk, pv), Q, pk, pv)


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("d,group,H,T", [(64, 32, 2, 2), (128, 128, 1, 7), (128, 32, 4, 16)])
@pytest.mark.parametrize("power", [20, 60])
def test_one_query_attends_to_what_the_others_do_not(fmt, d, group, H, T, power):
    """Queries of one tile with opposite signs: a row with large value scales has all the weight of some and none of the others'."""
    q, pk, pv, Q, ck, sk, cv, sv = cache(fmt, group, d, 2, 90, H, T, 202)
    score_row(ck, sk, 1, 11, Q, 60.0)
    sv[1, 11] *= 2.0 ** power
    Q[1::2] *= -1
    pk.set(ck, sk)
    pv.set(cv, sv)
    bounded(*attend(q, Q, pk, pv, n_rows=177), Q, pk, pv, 177)


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("d,group,T", [(64, 32, 1), (64, 64, 9), (128, 128, 1), (128, 32, 2), (128, 64, 10)])
@pytest.mark.parametrize("power", [12, 26, 60])
def test_large_values_come_and_go_along_the_rows(fmt, d, group, T, power):
    """Several units of rows to a warp: unattended rows with large value scales are met before, between and after the
    others, and a zero-valued row 12 above the rest (at most 2962 / 32 tiles of four heads over 29 splits or more: four units)."""
    q, pk, pv, Q, ck, sk, cv, sv = cache(fmt, group, d, 2, 1481, 40, T, 203)
    for row in range(5, 1481, 97):
        score_row(ck, sk, 0, row, Q, -80.0)
        sv[0, row] *= 2.0 ** power
    score_row(ck, sk, 1, 700, Q, 12.0)
    cv[1, 700] = 0.0
    pk.set(ck, sk)
    pv.set(cv, sv)
    bounded(*attend(q, Q, pk, pv), Q, pk, pv, units=4)
