"""Rows appended to pages of a quantised store that are in HBM slots already: every reader sees them, in stream order, and
the page is the same in both tiers."""
import ctypes
import math

import numpy as np
import pytest
import torch

import synth
from hsa_testlib import to_dev
from quant_testlib import Pages, attention64, encode

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import hybrid_sparse_attention_hkv_b200 as hsa
    from hybrid_sparse_attention_hkv_b200.store import QuantPageStore


def host_pages(store, kv):
    """The host tier of K or V as Pages, to read codes and scales from."""
    n = store.NP * store.page_bytes
    buf = (ctypes.c_uint8 * n).from_address(store.host[kv].host_ptr)
    p = Pages(hsa, store.quant, store.NP, store.rows, store.heads, store.head_dim, device="cpu", fill=0)
    p.raw = torch.from_numpy(np.frombuffer(buf, dtype=np.uint8).reshape(store.NP, store.page_bytes)).clone()
    return p


def clear_host(store):
    for h in store.host:
        ctypes.memset(h.host_ptr, 0, store.NP * store.page_bytes)


def check_both_tiers(store, pages):
    """Resident pages hold in their slots what the host tier holds, codes and scales."""
    sp, _ = store.residency()
    for kv, pool in ((0, store.slot_k), (1, store.slot_v)):
        host = host_pages(store, kv)
        for p in pages:
            slot = sp[p].item()
            assert slot >= 0
            raw = pool[slot].flatten().view(torch.uint8).cpu()
            assert torch.equal(raw[:host.code_bytes], host.raw[p, :host.code_bytes])
            end = host.off + host.scale_bytes
            assert torch.equal(raw[host.off:end], host.raw[p, host.off:end])


@pytest.mark.parametrize("fmt,group,d", [(0, 128, 128), (1, 32, 64), (2, 64, 128)])
@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("device_row", [False, True])
def test_rows_appended_to_resident_pages_are_read(fmt, group, d, rotated, device_row):
    NP, S, P, H = 5, 3, 60, 3
    quant = hsa.make_quant(fmt, group)
    store = QuantPageStore(quant, NP, S, P, H, d)
    try:
        clear_host(store)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        K, V = (to_dev(synth.normal_bf16((NP * P, H, d), 71, i)) for i in (1, 2))
        rope = hsa.make_rope(hsa.rope_freqs(d)[0].cuda(), hsa.ROPE_HALF) if rotated else None
        at = torch.arange(NP * P, dtype=torch.int32, device="cuda") if rotated else None
        written = torch.zeros(NP * P, dtype=torch.bool)

        def write(first, n):
            dev = torch.tensor([first - 7], dtype=torch.int64, device="cuda") if device_row else None
            store.write(K[first:first + n], V[first:first + n], 7 if device_row else first, ws, dev, rope,
                        at[first:first + n].contiguous() if rotated else None)
            written[first:first + n] = True

        write(0, 2 * P + 13)  # pages 0 and 1, and some of page 2
        sel = torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda")
        store.fetch(sel, ws)  # page 2 partly filled, page 3 empty
        residency = [x.tolist() for x in store.residency()]
        # one row; several; past the end of a resident page into the next resident one; into page 4, which is not
        # resident; again over rows of a page that is in its slot
        for first, n in ((2 * P + 13, 1), (2 * P + 14, 20), (2 * P + 34, P), (3 * P + 34, P), (5, 3)):
            write(first, n)
            assert [x.tolist() for x in store.residency()] == residency
            check_both_tiers(store, [0, 2, 3])
            k, v = (host_pages(store, kv).rows64() for kv in (0, 1))
            if not rotated:  # the host tier holds the rows that were written, and zeros
                for got, x in ((k, K), (v, V)):
                    codes, scales = encode(x.float().cpu(), fmt, group)
                    want = (codes.double().unflatten(-1, (-1, group)) * scales.double()[..., None]).flatten(-2)
                    assert torch.equal(got.flatten(0, 1), torch.where(written[:, None, None], want, 0.0))
            for pages in ([0, 2, 3], [2, 4], [1]):
                s = torch.tensor(pages, dtype=torch.int32, device="cuda")
                m = len(pages) * P
                Kc, Vc = (torch.zeros(m, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
                store.gather(s, Kc, Vc, ws)
                assert torch.equal(Kc.cpu(), k[pages].flatten(0, 1).float().bfloat16())
                assert torch.equal(Vc.cpu(), v[pages].flatten(0, 1).float().bfloat16())
        # a token over the appended rows
        Q = to_dev(synth.normal_bf16((1, H, d), 71, 3))
        out = torch.empty(1, H, d, device="cuda")
        aws = torch.zeros(hsa.hkv_attn_quant_workspace_size(1, H, H, d, 3, P), dtype=torch.uint8, device="cuda")
        store.attend(Q, sel, out, None, aws)
        kk, vv = (x[[0, 2, 3]].flatten(0, 1) for x in (k, v))
        want, _, mag = attention64(Q.double().cpu(), kk, vv, 1 / math.sqrt(d))
        bound = (2 * (mag * 2.0 ** -21 + 2.0 ** -22) + 2.0 ** -19) * vv.abs().amax()  # as the attention's own tests
        assert ((out.double().cpu() - want).abs() <= bound + 2.0 ** -24 * want.abs()).all()
        # a page that leaves its slot and comes back is the same
        store.fetch(torch.tensor([1, 4], dtype=torch.int32, device="cuda"), ws)
        store.fetch(sel, ws)
        check_both_tiers(store, [0, 2, 3])
        assert hsa.hsa_status_read(ws) == 0
    finally:
        store.close()


def test_sealing_a_resident_page_renews_its_slot():
    quant, NP, S, P, H, d = hsa.make_quant(1, 64), 3, 2, 32, 2, 64
    store = QuantPageStore(quant, NP, S, P, H, d)
    try:
        clear_host(store)
        ws = hsa.workspace(hsa.make_config(H, d, 8, 0, 64))
        kbar = torch.zeros(NP, H, d, device="cuda")
        K, V = (to_dev(synth.normal_bf16((P, H, d), 72, i)) for i in (1, 2))
        store.fetch(torch.tensor([1, 2], dtype=torch.int32, device="cuda"), ws)
        store.seal(1, K, V, kbar[1], ws)
        check_both_tiers(store, [1, 2])
        assert host_pages(store, 0).rows64()[1].abs().amax() > 0
        assert hsa.hsa_status_read(ws) == 0
    finally:
        store.close()


def test_a_captured_append_reaches_a_page_fetched_later():
    """Write, length and attention captured once: the replay after a fetch writes both tiers, with no new capture."""
    quant, NP, S, P, H, d = hsa.make_quant(0, 64), 2, 1, 40, 2, 64
    store = QuantPageStore(quant, NP, S, P, H, d)
    try:
        clear_host(store)
        ws = torch.zeros(hsa.hkv_attn_quant_workspace_size(1, H, H, d, 2, P), dtype=torch.uint8, device="cuda")
        Ks, Vs, Qs = (to_dev(synth.normal_bf16((60, H, d), 73, i)) for i in (1, 2, 3))
        k, v, x = (torch.zeros(1, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        row, n = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        sel = torch.arange(2, dtype=torch.int32, device="cuda")
        out = torch.empty(1, H, d, device="cuda")

        def step():
            store.write(k, v, 0, ws, row)
            store.attend(x, sel, out, None, ws, n)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for i in range(60):
            if i in (0, 17, 45):
                store.fetch(sel[i // 40:i // 40 + 1], ws)
            k.copy_(Ks[i:i + 1]), v.copy_(Vs[i:i + 1]), x.copy_(Qs[i:i + 1])
            row.fill_(i), n.fill_(i + 1)
            graph.replay()
            if i in (0, 16, 17, 39, 40, 44, 45, 59):
                rows = []
                for y in (Ks, Vs):
                    codes, scales = encode(y[:i + 1].float().cpu(), 0, 64)
                    rows.append((codes.double().unflatten(-1, (-1, 64)) * scales.double()[..., None]).flatten(-2))
                want, _, mag = attention64(Qs[i:i + 1].double().cpu(), *rows, 1 / math.sqrt(d))
                bound = (2 * (mag * 2.0 ** -21 + 2.0 ** -22) + 2.0 ** -19) * rows[1].abs().amax()
                assert ((out.double().cpu() - want).abs() <= bound + 2.0 ** -24 * want.abs()).all(), i
        assert hsa.hsa_status_read(ws) == 0
    finally:
        store.close()
