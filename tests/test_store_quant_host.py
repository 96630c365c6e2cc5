"""The store of quantised pages on a machine without a GPU: refusals of its writing call (none reaches the CUDA runtime)."""
import ctypes

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


def rows(data=A, H=2, ts=128, hs=64):
    return hsa._pack_rows(data or 0, H, ts, hs)


def store(NP=4, S=2, P_tok=None, H=4, d=128, host=A, slot=A, state=A, quant=(0, 64), geometry=(8, 2, 64)):
    if P_tok is None:
        P_tok = hsa.hkv_quant_page_size(hsa.make_quant(*quant), *geometry)[0] // 1024
    return hsa.StoreDesc(NP, S, P_tok, H, d, host, host, slot, slot, state)


def call(lib, st=None, q=(0, 64), K=None, V=None, T=4, d=64, dtype=0, rope=None, pos=None, P_tok=8, first=0, dev=None, ws=WS, wsb=256):
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    st = store() if st is None else st
    return lib.hkv_store_write_quant(ref(st) if st else None, ref(hsa.make_quant(*q)) if q else None, K or rows(), V or rows(), T, d,
                                     dtype, rope, pos, 4, P_tok, first, dev, ws, wsb, None)


def test_store_write_refusals(lib):
    rope = hsa.make_rope(hsa.rope_freqs(64)[0])
    bad = [
        (dict(st=False), 1), (dict(st=store(NP=0)), 1), (dict(st=store(host=0)), 1), (dict(st=store(slot=MIS)), 1),
        (dict(st=store(state=0)), 1), (dict(st=store(state=A + 16)), 1), (dict(q=None), 1), (dict(q=(3, 64)), 1), (dict(q=(0, 128)), 1),
        (dict(T=-1), 1), (dict(dtype=3), 1), (dict(d=32), 2), (dict(K=rows(data=None)), 1), (dict(V=rows(H=3)), 1),
        (dict(rope=rope.ref), 1), (dict(P_tok=0), 1), (dict(first=-1), 1), (dict(first=29), 1), (dict(first=2 ** 62, dev=P(A)), 1),
        (dict(dev=P(MIS)), 1), (dict(ws=None), 3), (dict(wsb=255), 3),
        # a store whose pages have another size: of bf16, of another format, of other rows or heads
        (dict(st=store(P_tok=16, H=2, d=64)), 1), (dict(q=(2, 64)), 1), (dict(P_tok=16), 1), (dict(K=rows(H=4, ts=256), V=rows(H=4, ts=256)), 1),
    ]
    for kw, code in bad:
        assert call(lib, **kw) == code, (kw, lib.hsa_last_error_detail().decode())
    assert call(lib, T=0, K=rows(data=None), V=rows(data=None)) == 0
    with hsa.injected_fault(hsa.FAULT_LAUNCH):
        for kw in (dict(first=28), dict(first=-3, dev=P(A)), dict(rope=rope.ref, pos=P(A))):
            assert call(lib, **kw) == 4, (kw, lib.hsa_last_error_detail().decode())
    with hsa.injected_fault(hsa.FAULT_WORKSPACE):
        assert call(lib) == 3


def test_binding_of_the_store_write_checks_its_tensors(lib):
    quant, desc = hsa.make_quant(0, 64), store()
    x, ws = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.uint8)
    pos = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(hsa.HsaError, match="CUDA device"):
        hsa.hkv_store_write_quant(desc, quant, x, x, 8, 0, ws)
    for bad in (lambda: hsa.hkv_store_write_quant(desc, quant, x.double(), x, 8, 0, ws),
                lambda: hsa.hkv_store_write_quant(desc, quant, x, x[:3], 8, 0, ws),
                lambda: hsa.hkv_store_write_quant(desc, quant, x, x, 8, 0, ws.int()),
                lambda: hsa.hkv_store_write_quant(desc, quant, x, x, 8, 0, ws, pos=pos),
                lambda: hsa.hkv_store_write_quant(desc, quant, x, x, 8, 0, ws, first_row_dev=pos)):
        with pytest.raises(hsa.HsaError) as e:
            bad()
        assert e.value.code == 1
