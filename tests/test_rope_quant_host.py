"""Rotary positions and quantised pages on a machine without a GPU: the host-side helpers against their formulas, and
every refusal (none of these calls reaches the CUDA runtime)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import hybrid_sparse_attention_hkv_b200 as hsa

P = ctypes.c_void_p
A, MIS = 0x10000, 0x10004
WS = P(0x100000)


@pytest.fixture(scope="module")
def lib():
    from hybrid_sparse_attention_hkv_b200 import build
    build.build()
    return hsa.load_library()


def detail():
    return hsa.load_library().hsa_last_error_detail().decode()


def test_frequencies_follow_their_formulas(lib):
    dim, base, factor, ctx = 64, 10000.0, 4.0, 4096
    i = np.arange(dim // 2)
    plain = base ** (-2.0 * i / dim)
    f, m = hsa.rope_freqs(dim, base)
    np.testing.assert_allclose(f.numpy(), plain, rtol=1e-14)
    assert m == 1.0
    f, m = hsa.rope_freqs(dim, base, hsa.ROPE_SCALE_LINEAR, factor)
    np.testing.assert_allclose(f.numpy(), plain / factor, rtol=1e-14)
    f, m = hsa.rope_freqs(dim, base, hsa.ROPE_SCALE_NTK, factor)
    np.testing.assert_allclose(f.numpy(), (base * factor ** (dim / (dim - 2))) ** (-2.0 * i / dim), rtol=1e-13)
    # the slowest pair is stretched by exactly the factor
    assert math.isclose(f[-1], plain[-1] / factor, rel_tol=1e-12) and f[0] == 1.0
    f, m = hsa.rope_freqs(dim, base, hsa.ROPE_SCALE_YARN, factor, ctx)
    turns = ctx * plain / (2 * math.pi)
    keep = np.clip(np.log(turns) / np.log(32.0), 0, 1)
    np.testing.assert_allclose(f.numpy(), plain * keep + plain / factor * (1 - keep), rtol=1e-13)
    assert keep[0] == 1 and keep[-1] == 0 and ((keep > 0) & (keep < 1)).any()
    assert m == np.float32(0.1 * math.log(factor) + 1)
    assert hsa.rope_freqs(2)[0].tolist() == [1.0]


@pytest.mark.parametrize("kw", [dict(dim=0), dict(dim=7), dict(dim=-2), dict(dim=64, base=1.0), dict(dim=64, base=float("nan")),
                                dict(dim=64, scaling=9), dict(dim=64, scaling=1, factor=0.5),
                                dict(dim=64, scaling=1, factor=float("inf")), dict(dim=2, scaling=2, factor=2.0),
                                dict(dim=64, scaling=3, factor=2.0, orig_context=0)])
def test_frequency_refusals(lib, kw):
    with pytest.raises(hsa.HsaError) as e:
        hsa.rope_freqs(**kw)
    assert e.value.code == 1


@pytest.mark.parametrize("fmt,group,P_tok,H,d", [(0, 128, 12480, 40, 128), (1, 32, 7, 3, 64), (2, 64, 1, 1, 128), (2, 32, 5, 1, 64)])
def test_page_size(lib, fmt, group, P_tok, H, d):
    n, off = hsa.hkv_quant_page_size(hsa.make_quant(fmt, group), P_tok, H, d)
    codes = P_tok * H * d // (2 if fmt == 2 else 1)
    assert off % 256 == 0 and codes <= off < codes + 256
    need = off + 4 * P_tok * H * d // group
    assert n % 1024 == 0 and need <= n < need + 1024


@pytest.mark.parametrize("q,P_tok,H,d,code", [((3, 128), 8, 1, 128, 1), ((0, 16), 8, 1, 128, 2), ((0, 128), 8, 1, 64, 1),
                                              ((0, 64), 0, 1, 64, 1), ((0, 64), 8, 0, 64, 1), ((0, 32), 8, 1, 96, 2),
                                              ((0, 64), 8, 16385, 64, 2)])
def test_page_refusals(lib, q, P_tok, H, d, code):
    with pytest.raises(hsa.HsaError) as e:
        hsa.hkv_quant_page_size(hsa.make_quant(*q), P_tok, H, d)
    assert e.value.code == code


def rope_struct(**kw):
    v = dict(layout=0, rot=64, axes=(32,), mscale=1.0, inv=A) | kw
    return hsa._Rope(v["layout"], v["rot"], len(v["axes"]), (ctypes.c_int * 3)(*v["axes"]), v["mscale"], v["inv"])


class Rows(ctypes.Structure):  # hsa_rows_t
    _fields_ = [("data", ctypes.c_void_p), ("H", ctypes.c_int), ("token_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong)]


def rows(**kw):
    v = dict(data=A, H=2, ts=128, hs=64) | kw
    return Rows(v["data"], v["H"], v["ts"], v["hs"])


def test_the_binding_packs_rows_as_the_structure():
    t = torch.zeros(5, 4, 64, dtype=torch.float16)[:, 1:3]
    assert hsa._rows(t, "t", "here", -1, torch.float16, 5, 64) == bytes(Rows(t.data_ptr(), 2, 256, 64))
    assert hsa._rows(t[:1, :1], "t", "here", -1, torch.float16, 1, 64) == bytes(Rows(t.data_ptr(), 1, 64, 64))


def call_rope(lib, fn="hsa_rope", rope=None, pos=A, pos_stride=4, T=4, d=64, dtype=0, qi=None, qo=None, ki=None, ko=None):
    ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
    rope = rope_struct() if rope is None else rope
    return getattr(lib, fn)(ref(rope) if rope else None, P(pos) if pos else None, pos_stride, T, d, dtype, ref(qi or rows()),
                            ref(qo or rows()), ref(ki), ref(ko), None)


@pytest.mark.parametrize("fn", ["hsa_rope", "hsa_rope_bwd"])
def test_rope_refusals(lib, fn):
    bad = [
        (dict(rope=False), 1), (dict(T=-1), 1), (dict(dtype=3), 1), (dict(d=96), 2), (dict(d=0), 1), (dict(pos=None), 1), (dict(pos=0x10002), 1),
        (dict(rope=rope_struct(layout=2)), 1), (dict(rope=rope_struct(rot=80, axes=(40,))), 1),
        (dict(rope=rope_struct(rot=24, axes=(12,))), 2), (dict(rope=rope_struct(rot=0, axes=(0,))), 1),
        (dict(rope=rope_struct(axes=(31,))), 1), (dict(rope=rope_struct(axes=(16, 17))), 1),
        (dict(rope=rope_struct(axes=(40, -8))), 1), (dict(rope=rope_struct(axes=(2 ** 31 - 1, 2 ** 31 - 1, 34))), 1),
        (dict(rope=rope_struct(mscale=float("nan"))), 1), (dict(rope=rope_struct(inv=None)), 1), (dict(rope=rope_struct(inv=MIS)), 1),
        (dict(rope=rope_struct(axes=(16, 16)), pos_stride=3), 1),
        (dict(qi=rows(data=None)), 1), (dict(qi=rows(data=0x10002)), 1), (dict(qi=rows(ts=132)), 1), (dict(qi=rows(hs=60)), 1),
        (dict(qi=rows(hs=56)), 1), (dict(qi=rows(ts=-128)), 1), (dict(qo=rows(ts=0)), 1), (dict(qo=rows(ts=64)), 1),
        (dict(qo=rows(ts=128, hs=128)), 1), (dict(qo=rows(ts=64, hs=192)), 1), (dict(qo=rows(H=3)), 1), (dict(qi=rows(H=0)), 1),
        (dict(qi=rows(H=16385), qo=rows(H=16385)), 2),
        (dict(ki=rows()), 1), (dict(ki=rows(), ko=rows(H=1)), 1), (dict(ki=rows(), ko=rows(ts=0)), 1),
    ]
    for kw, code in bad:
        assert call_rope(lib, fn, **kw) == code, (kw, detail())
        assert detail().startswith(fn + ":"), (kw, detail())
    r = rope_struct()
    r.n_axes = 4
    assert call_rope(lib, fn, rope=r) == 1
    # nothing to do: accepted without pointers, shapes still checked
    assert call_rope(lib, fn, T=0, pos=None, qi=rows(data=None), qo=rows(data=None)) == 0
    assert call_rope(lib, fn, T=0, d=96) == 2
    with hsa.injected_fault(hsa.FAULT_LAUNCH):
        assert call_rope(lib, fn) == 4 and "injected" in detail()
        # fp32 strides count in 4-byte elements, a broadcast input row is allowed
        assert call_rope(lib, fn, dtype=2, qi=rows(ts=132, hs=64), qo=rows(ts=132)) == 4
        assert call_rope(lib, fn, qi=rows(data=0x20000, ts=0)) == 4
        assert call_rope(lib, fn, qo=rows(data=0x20000, ts=64, hs=256)) == 4  # [H, T, d]


@pytest.mark.parametrize("fn", ["hsa_rope", "hsa_rope_bwd"])
def test_rope_refuses_outputs_over_other_elements(lib, fn):
    B = 0x20000
    for kw in (dict(qi=rows(ts=0)), dict(qi=rows(ts=256)), dict(qo=rows(ts=64, hs=256)),     # one address, other strides
               dict(ki=rows(data=B), ko=rows(data=B, ts=256)),
               dict(ki=rows(data=B), ko=rows()), dict(qo=rows(data=B), ki=rows(data=B), ko=rows(data=0x30000)),
               dict(qi=rows(data=0x30000), qo=rows(data=B), ki=rows(data=0x40000), ko=rows(data=B))):
        assert call_rope(lib, fn, **kw) == 1 and "one address" in detail(), kw
    with hsa.injected_fault(hsa.FAULT_LAUNCH):
        # in place; queries and keys of one buffer; one row whatever its stride; one head whatever its stride; shared inputs
        for kw in (dict(ki=rows(data=B), ko=rows(data=B)), dict(ki=rows(data=A + 256, ts=256), ko=rows(data=A + 256, ts=256)),
                   dict(T=1, qi=rows(ts=0)), dict(qi=rows(H=1, hs=64), qo=rows(H=1, hs=128)),
                   dict(qo=rows(data=B), ki=rows(), ko=rows(data=0x30000))):
            assert call_rope(lib, fn, **kw) == 4, (kw, detail())


def call_rows(lib, q=(0, 64), K=None, V=None, T=4, d=64, dtype=0, rope=None, pos=None, pos_stride=4, pk=P(A), pv=P(A), NP=2,
              P_tok=8, first=0, dev=None, ws=WS, wsb=256):
    ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
    return lib.hkv_quant_rows(ref(hsa.make_quant(*q)) if q else None, ref(K or rows()), ref(V or rows()), T, d, dtype, ref(rope),
                              pos, pos_stride, pk, pv, NP, P_tok, first, dev, ws, wsb, None)


def test_quant_rows_refusals(lib):
    bad = [
        (dict(q=None), 1), (dict(q=(5, 64)), 1), (dict(q=(0, 128)), 1), (dict(q=(0, 48)), 2), (dict(T=-1), 1), (dict(dtype=-1), 1),
        (dict(d=32), 2), (dict(K=rows(data=None)), 1), (dict(V=rows(H=3)), 1), (dict(V=rows(ts=4)), 1), (dict(rope=rope_struct()), 1),
        (dict(pk=None), 1), (dict(pv=None), 1), (dict(NP=0), 1), (dict(P_tok=0), 1), (dict(first=-1), 1), (dict(first=13), 1),
        (dict(first=2 ** 62), 1), (dict(first=2 ** 62, dev=P(A)), 1), (dict(dev=P(MIS)), 1), (dict(ws=None), 3), (dict(wsb=255), 3),
        (dict(ws=P(0x100010)), 3),
    ]
    for kw, code in bad:
        assert call_rows(lib, **kw) == code, (kw, detail())
    assert call_rows(lib, T=0, K=rows(data=None), V=rows(data=None)) == 0
    with hsa.injected_fault(hsa.FAULT_LAUNCH):
        for kw in (dict(first=12), dict(first=-3, dev=P(A)), dict(rope=rope_struct(), pos=P(A))):
            assert call_rows(lib, **kw) == 4, (kw, detail())
    with hsa.injected_fault(hsa.FAULT_WORKSPACE):
        assert call_rows(lib) == 3
    with hsa.injected_fault(hsa.FAULT_ARG):
        assert call_rows(lib) == 1


def call_gather(lib, q=(0, 64), pk=P(A), pv=P(A), NP=4, sel=P(A), Kp=2, P_tok=8, H=2, d=64, rope=None, pos=None, pos_stride=16,
                Kc=P(A), Vc=P(A), kb=None, ws=WS, wsb=256):
    return lib.hkv_gather_quant(ctypes.byref(hsa.make_quant(*q)), pk, pv, NP, sel, Kp, P_tok, H, d,
                                None if rope is None else ctypes.byref(rope), pos, pos_stride, Kc, Vc, kb, ws, wsb, None)


def test_gather_quant_refusals(lib):
    bad = [
        (dict(q=(-1, 64)), 1), (dict(q=(1, 128)), 1), (dict(pk=None), 1), (dict(pv=None), 1), (dict(NP=0), 1), (dict(sel=None), 1),
        (dict(Kp=0), 1), (dict(Kp=5), 1), (dict(P_tok=0), 1), (dict(H=0), 1), (dict(d=256), 2), (dict(Kc=None), 1),
        (dict(Vc=P(0x10008)), 1), (dict(kb=P(MIS)), 1), (dict(P_tok=2 ** 30), 2), (dict(rope=rope_struct()), 1),
        (dict(rope=rope_struct(axes=(16, 16)), pos=P(A), pos_stride=15), 1), (dict(ws=None), 3), (dict(wsb=0), 3),
    ]
    for kw, code in bad:
        assert call_gather(lib, **kw) == code, (kw, detail())
    with hsa.injected_fault(hsa.FAULT_LAUNCH):
        assert call_gather(lib, rope=rope_struct(axes=(16, 16)), pos=P(A), kb=P(A)) == 4


def call_attn(lib, q=(0, 64), Q=P(A), T=2, Hq=4, pk=P(A), pv=P(A), NP=4, sel=P(A), Kp=2, P_tok=8, H=2, d=64, n=None, scale=0.0,
              out=P(A), lse=None, ws=WS, wsb=1 << 24):
    return lib.hkv_attn_quant(ctypes.byref(hsa.make_quant(*q)), Q, T, Hq, pk, pv, NP, sel, Kp, P_tok, H, d, n, scale, out, 0, lse, ws,
                              wsb, None)


def test_attn_quant_refusals(lib):
    bad = [
        (dict(q=(0, 7)), 2), (dict(T=-1), 1), (dict(T=65), 2), (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(T=64, Hq=16384, H=1), 2), (dict(Hq=16386, H=2), 2), (dict(H=0), 1), (dict(Kp=0), 1),
        (dict(Kp=5), 1), (dict(NP=0), 1), (dict(P_tok=0), 1), (dict(P_tok=2 ** 30), 2), (dict(d=80), 2), (dict(Q=None), 1),
        (dict(Q=P(MIS)), 1), (dict(out=None), 1), (dict(pk=None), 1), (dict(sel=None), 1), (dict(scale=float("nan")), 1),
        (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1), (dict(ws=None), 3), (dict(wsb=255), 3), (dict(Kp=4, P_tok=4096, wsb=4096), 3),
    ]
    for kw, code in bad:
        assert call_attn(lib, **kw) == code, (kw, detail())
    assert call_attn(lib, T=0, Q=None, out=None) == 0
    with hsa.injected_fault(hsa.FAULT_LAUNCH):
        assert call_attn(lib) == 4
    small = hsa.hkv_attn_quant_workspace_size(1, 1, 1, 64, 1, 16)
    big = hsa.hkv_attn_quant_workspace_size(16, 40, 40, 128, 4, 12480)
    assert small == 256 and big > small and big % 256 == 0
    with pytest.raises(hsa.HsaError):
        hsa.hkv_attn_quant_workspace_size(65, 1, 1, 64, 1, 16)


def test_a_step_refuses_a_store_of_other_pages():
    """Reading pages of one format as another's runs over their ends, so the step looks before it allocates anything."""
    from hybrid_sparse_attention_hkv_b200.step import HkvHsaStep
    from hybrid_sparse_attention_hkv_b200.store import PageStore, QuantPageStore
    held = QuantPageStore.__new__(QuantPageStore)
    held.quant, held.NP, held.rows, held.heads, held.head_dim = hsa.make_quant(0, 64), 4, 256, 2, 64
    plain = PageStore.__new__(PageStore)

    def step(store, quant, H=2, d=64, P_tok=256, NP=4):
        return HkvHsaStep(H, d, 256, P_tok, NP, 2, 64, None, None, device="cpu", store=store, quant=quant)
    for store, quant, kw in ((held, None, {}), (plain, hsa.make_quant(0, 64), {}), (held, hsa.make_quant(1, 64), {}),
                             (held, hsa.make_quant(0, 32), {}), (held, hsa.make_quant(0, 64), dict(P_tok=512)),
                             (held, hsa.make_quant(0, 64), dict(H=4)), (held, hsa.make_quant(0, 64), dict(d=128)),
                             (held, hsa.make_quant(0, 64), dict(NP=8))):
        with pytest.raises(ValueError, match="store's pages"):
            step(store, quant, **kw)


def test_a_closed_quantised_store_is_not_read_or_written():
    from hybrid_sparse_attention_hkv_b200.store import QuantPageStore
    s = QuantPageStore.__new__(QuantPageStore)
    s._own, s.host = False, (None, None)
    s.quant, s.NP, s.rows, s.heads, s.head_dim = hsa.make_quant(0, 64), 2, 4, 1, 64
    s.close()
    x = torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    sel, ws = torch.zeros(1, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    for call in (lambda: s.write(x, x, 0, ws), lambda: s.seal(0, x, x, x, ws), lambda: s.gather(sel, x, x, ws),
                 lambda: s.attend(x, sel, x, None, ws)):
        with pytest.raises(hsa.HsaError, match="closed"):
            call()


def test_the_longest_caches_are_split_like_long_ones(lib):
    size = lambda *a: hsa.hkv_attn_quant_workspace_size(1, 2, 2, 64, *a)  # noqa: E731
    assert size(1, 2 ** 31 - 1) == size(1, 2 ** 31 - 1024) == size(2 ** 31 - 1, 1) == size(2 ** 20, 2 ** 10) > 256


def test_tables_selections_and_lengths_are_aligned(lib):
    ODD = P(0x10002)
    for kw in (dict(pk=P(MIS)), dict(pv=P(MIS))):
        assert call_rows(lib, **kw) == 1 and "aligned" in detail(), kw
        assert call_gather(lib, **kw) == 1 and "aligned" in detail(), kw
        assert call_attn(lib, **kw) == 1 and "aligned" in detail(), kw
    assert call_gather(lib, sel=ODD) == 1 and "aligned" in detail()
    for kw in (dict(sel=ODD), dict(n=ODD), dict(lse=ODD)):
        assert call_attn(lib, **kw) == 1 and "aligned" in detail(), kw
    with hsa.injected_fault(hsa.FAULT_LAUNCH):  # 4 bytes are enough for a selection, a length and an lse
        assert call_gather(lib, sel=P(MIS)) == 4
        assert call_attn(lib, sel=P(MIS), n=P(MIS), lse=P(MIS)) == 4


def test_binding_refuses_what_the_library_cannot_see(lib):
    """Types, shapes, strides and devices of the tensors are checked before their addresses are taken."""
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    inv, _ = hsa.rope_freqs(64)
    rope = hsa.make_rope(inv)
    pos = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(hsa.HsaError, match="CUDA device"):
        hsa.hsa_rope(rope, pos, q, q.clone())
    cases = [
        lambda: hsa.hsa_rope(rope, pos, q.double(), q),
        lambda: hsa.hsa_rope(rope, pos, q, q.float()),
        lambda: hsa.hsa_rope(rope, pos, q, q[:3]),
        lambda: hsa.hsa_rope(rope, pos, q, q.transpose(1, 2)),
        lambda: hsa.hsa_rope(rope, pos.long(), q, q),
        lambda: hsa.hsa_rope(rope, pos[:3], q, q),
        lambda: hsa.hsa_rope(rope, None, q, q),
        lambda: hsa.hsa_rope(rope, pos, q, q, k=q),
        lambda: hsa.hsa_rope(rope, pos, q[..., ::2], q[..., ::2]),
        lambda: hsa.make_rope(inv.float()),
        lambda: hsa.make_rope(inv, axis_pairs=[16, 15]),
        lambda: hsa.make_rope(inv, axis_pairs=[8, 8, 8, 8]),
        lambda: hsa.make_rope(inv[::2], axis_pairs=[16]),
    ]
    quant = hsa.make_quant(0, 64)
    table, ws = torch.zeros(2, dtype=torch.int64), torch.zeros(256, dtype=torch.uint8)
    sel, kc = torch.zeros(1, dtype=torch.int32), torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    cases += [
        lambda: hsa.hkv_quant_rows(quant, q, q[:, :1].float(), table, table, 8, 0, ws),
        lambda: hsa.hkv_quant_rows(quant, q, q, table, table[:1], 8, 0, ws),
        lambda: hsa.hkv_quant_rows(quant, q, q, table.int(), table, 8, 0, ws),
        lambda: hsa.hkv_quant_rows(quant, q, q, table, table, 8, 0, ws, first_row_dev=torch.zeros(1)),
        lambda: hsa.hkv_quant_rows(quant, q, q, table, table, 8, 0, ws, first_row_dev=torch.zeros(2, dtype=torch.int64)),
        lambda: hsa.hkv_quant_rows(quant, q, q, table, table, 8, 0, ws, pos=pos),
        lambda: hsa.hkv_gather_quant(quant, table, table, sel, 1, 8, 2, 64, kc, kc[:7], ws),
        lambda: hsa.hkv_gather_quant(quant, table, table, sel.long(), 1, 8, 2, 64, kc, kc, ws),
        lambda: hsa.hkv_gather_quant(quant, table, table, sel, 1, 8, 2, 64, kc, kc, ws, kbar128=torch.zeros(2, 2, 64)),
        lambda: hsa.hkv_gather_quant(quant, table, table, sel, 1, 8, 2, 64, kc, kc, ws, rope=rope, pos=pos),
        lambda: hsa.hkv_attn_quant(quant, q.float(), table, table, sel, 1, 8, 2, kc, None, ws),
        lambda: hsa.hkv_attn_quant(quant, q, table, table, sel, 1, 8, 2, q.half(), None, ws),
        lambda: hsa.hkv_attn_quant(quant, q, table, table, sel, 1, 8, 2, q[:3], None, ws),
        lambda: hsa.hkv_attn_quant(quant, q, table, table, sel, 1, 8, 2, q, torch.zeros(4, 3), ws),
    ]
    for i, call in enumerate(cases):
        with pytest.raises(hsa.HsaError) as e:
            call()
        assert e.value.code == 1, i
