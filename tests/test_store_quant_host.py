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


class FreedHost:
    """A host tier that can be freed once."""

    def __init__(self):
        self.dev_ptr, self.freed = A, 0

    def close(self):
        self.freed += 1


def a_store(kind, own=False):
    """A store object without its device memory."""
    s = kind.__new__(kind)
    s._own, s.host = own, (FreedHost(), FreedHost())
    s.desc, s.NP, s.S, s.table_k, s.table_v = store(), 4, 2, 0, 0
    s.quant, s.rows, s.heads, s.head_dim = hsa.make_quant(0, 64), 8, 2, 64
    s.state = s.slot_k = torch.zeros(256, dtype=torch.uint8)
    return s


@pytest.mark.parametrize("quantised", [False, True])
def test_a_closed_store_neither_copies_nor_gives_its_tables(lib, quantised):
    """Their kernels and readers would go to host memory that is gone."""
    from hybrid_sparse_attention_hkv_b200.store import PageStore, QuantPageStore
    s = a_store(QuantPageStore if quantised else PageStore)
    s.close()
    sel, ws, x = torch.zeros(1, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8), torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: s.fetch(sel, ws), lambda: s.prefetch(torch.zeros(4), None, 1, ws), lambda: s.page_tables(),
                 lambda: s.seal(0, x, x, torch.zeros(2, 64), ws)):
        with hsa.injected_fault(hsa.FAULT_LAUNCH):  # nothing is launched whatever the call does
            with pytest.raises(hsa.HsaError, match="closed"):
                call()


def test_a_store_is_closed_once(monkeypatch):
    from hybrid_sparse_attention_hkv_b200.store import QuantPageStore
    waited = []
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: waited.append(device))
    s = a_store(QuantPageStore, own=True)
    held = s.host
    s.close()
    s.close()
    assert [h.freed for h in held] == [1, 1]
    assert len(waited) == 1  # kernels on their way through the host tier end before it goes


@pytest.mark.parametrize("quantised", [False, True])
def test_a_step_over_a_closed_store_launches_nothing(monkeypatch, quantised):
    """The step kept the store's tables: it looks before its first launch."""
    from hybrid_sparse_attention_hkv_b200 import step as module
    from hybrid_sparse_attention_hkv_b200.store import PageStore, QuantPageStore
    s = a_store(QuantPageStore if quantised else PageStore)
    st = module.HkvHsaStep.__new__(module.HkvHsaStep)
    st.store, st.out, st.rope = s, None, None
    s.close()

    def launched(*a, **k):
        raise AssertionError("launched")
    for name in ("hkv_select_pages", "hkv_select_prompt", "hkv_gather", "hkv_gather_quant", "hkv_block_means_from_pages"):
        monkeypatch.setattr(module, name, launched)
    st.kbar_pages = st.Kp = st.sel = st.ws = st.scores = st.seg = st.cand_range = None
    for call in (lambda: st(None, None, None, None, None, None, None), lambda: st.prepare_chunk(None, None, None),
                 lambda: st(None, None, None, None, None, None, None, e_cur=0), lambda: st.prepare_chunk(None, None, None, e_cur=0)):
        with pytest.raises(hsa.HsaError, match="closed"):
            call()


def test_a_quantised_store_has_the_shape_of_its_pages(lib, monkeypatch):
    """P_tok, H and d are the rows', heads' and columns' of its pages, as a PageStore's; the block of bytes that its residency
    calls move is the descriptor's."""
    from hybrid_sparse_attention_hkv_b200 import store as module

    def no_memory(self, NP, S, P_tok, H, d, host=None, stream=None):
        self.NP, self.S, self.P_tok, self.H, self.d, self.host = NP, S, P_tok, H, d, (FreedHost(), FreedHost())
        self.slot_k = torch.zeros(1)
        self.desc = store(NP, S, P_tok, H, d)
    monkeypatch.setattr(module.PageStore, "__init__", no_memory)
    s = module.QuantPageStore(hsa.make_quant(1, 32), 5, 2, 200, 3, 128)
    assert (s.NP, s.S, s.P_tok, s.H, s.d) == (5, 2, 200, 3, 128) == (s.NP, s.S, s.rows, s.heads, s.head_dim)
    assert s.desc.P_tok * s.desc.H * s.desc.d * 2 == s.page_bytes == hsa.hkv_quant_page_size(s.quant, 200, 3, 128)[0]


def test_rows_on_another_device_than_the_store_are_refused(lib):
    """Its tables are in the memory of its own device."""
    from hybrid_sparse_attention_hkv_b200.store import QuantPageStore

    class OnAnother:
        device = "cuda:1"

        def get_device(self):
            return 1
    s = a_store(QuantPageStore)
    x, ws = torch.zeros(8, 2, 64, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.uint8)
    s.slot_k = OnAnother()
    for call in (lambda: s.write(x, x, 0, ws), lambda: s.seal(0, x, x, torch.zeros(2, 64), ws)):
        with pytest.raises(hsa.HsaError, match="K is on cpu, the store on cuda:1"):
            call()
