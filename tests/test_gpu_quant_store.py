"""Quantised pages in the tiered store and in the step: rows written through the mapped host tier, residency as the plain
model's, the active cache read from either tier, a few tokens attending to the pages, and a whole step over them."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import synth
from hsa_testlib import assert_close, bits_of, check_selection, selection_lists, to_dev
from oracle.store import PageStoreModel
from quant_testlib import HALF_STEP, Pages, attention64, encode, rope64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import hybrid_sparse_attention_hkv_b200 as hsa
    from hybrid_sparse_attention_hkv_b200.step import HkvHsaStep
    from hybrid_sparse_attention_hkv_b200.store import QuantPageStore


def host_bytes(store, kv):
    n = store.NP * store.page_bytes
    buf = (ctypes.c_uint8 * n).from_address(store.host[kv].host_ptr)
    return torch.from_numpy(np.frombuffer(buf, dtype=np.uint8).reshape(store.NP, store.page_bytes))


def as_pages(store, raw):
    """`raw` [n, page_bytes] as Pages, to read codes and scales from."""
    p = Pages(hsa, store.quant, raw.shape[0], store.rows, store.heads, store.head_dim, device="cpu", fill=0)
    p.raw = raw
    return p


@pytest.mark.parametrize("fmt,group", [(0, 128), (1, 32), (2, 64)])
def test_store_of_quantised_pages(fmt, group):
    NP, S, P, H, d = 6, 3, 200, 3, 128
    quant = hsa.make_quant(fmt, group)
    store = QuantPageStore(quant, NP, S, P, H, d)
    try:
        ws = hsa.workspace(hsa.make_config(H, d, 8, 0, 64))
        kbar = torch.zeros(NP, H, d, device="cuda")
        K, V = (to_dev(synth.normal_bf16((NP, P, H, d), 61, i)) for i in (1, 2))
        for p in range(NP - 1):
            store.seal(p, K[p], V[p], kbar[p], ws)
        for t in range(0, P, 77):  # the last page row by row, as a chunk at a time
            store.write(K[NP - 1, t:t + 77], V[NP - 1, t:t + 77], (NP - 1) * P + t, ws)
        torch.cuda.synchronize()
        ref = np.stack([oracle.page_summary(bits_of(K[p])) for p in range(NP - 1)])
        np.testing.assert_allclose(kbar[:NP - 1].cpu().numpy(), ref, rtol=1e-5, atol=1e-6)
        rows = []
        for kv, x in ((0, K), (1, V)):
            codes, scales = encode(x.float().cpu(), fmt, group)
            got = as_pages(store, host_bytes(store, kv))
            assert torch.equal(got.codes(), codes) and torch.equal(got.scales(), scales)
            rows.append(got.rows64())
        model = PageStoreModel(NP, S)
        Q = to_dev(synth.normal_bf16((2, H, d), 61, 3))
        for sel in ([0, 2, 5], [1, 2, 3], [5], [0, 4, 5]):
            s = torch.tensor(sel, dtype=torch.int32, device="cuda")
            n = len(sel) * P
            k, v = (r[sel].flatten(0, 1) for r in rows)
            out = torch.empty(2, H, d, device="cuda")
            aws = torch.zeros(hsa.hkv_attn_quant_workspace_size(2, H, H, d, len(sel), P), dtype=torch.uint8, device="cuda")
            for resident in (False, True):  # from the host tier first, then from the slots
                if resident:
                    model.fetch(sel)
                    store.fetch(s, ws)
                    sp, ps = store.residency()
                    assert sp.cpu().tolist() == model.slot_of_page and ps.cpu().tolist() == model.page_of_slot
                Kc, Vc = (torch.zeros(n, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
                store.gather(s, Kc, Vc, ws)
                assert torch.equal(Kc.cpu(), k.float().bfloat16()) and torch.equal(Vc.cpu(), v.float().bfloat16())
                store.attend(Q, s, out, None, aws)
                want, _, mag = attention64(Q.double().cpu(), k, v, 1 / math.sqrt(d))
                bound = (2 * (mag * 2.0 ** -21 + 2.0 ** -22) + 2.0 ** -19) * v.abs().amax()  # as the attention's own tests
                assert ((out.double().cpu() - want).abs() <= bound + 2.0 ** -24 * want.abs()).all()
            for slot, p in enumerate(model.page_of_slot):
                if p >= 0:  # the whole block of the page, codes and scales
                    for kv, pool in ((0, store.slot_k), (1, store.slot_v)):
                        raw = pool[slot].flatten().view(torch.uint8).cpu()
                        used = as_pages(store, host_bytes(store, kv)[p:p + 1])
                        end = used.off + used.scale_bytes
                        assert torch.equal(raw[:used.code_bytes], used.raw[0, :used.code_bytes])
                        assert torch.equal(raw[used.off:end], used.raw[0, used.off:end])
        scores = torch.tensor([0.1, 5.0, 3.0, -math.inf, 4.0, 2.0], device="cuda")
        keep = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
        model.prefetch(scores.cpu().double().numpy(), [0, 5], 1)
        store.prefetch(scores, keep, 1, ws)
        sp, ps = store.residency()
        assert sp.cpu().tolist() == model.slot_of_page and ps.cpu().tolist() == model.page_of_slot
        assert hsa.hsa_status_read(ws) == 0 and hsa.hsa_status_read(aws) == 0
        for bad in (lambda: store.seal(NP, K[0], V[0], kbar[0], ws), lambda: store.seal(0, K[0, :7], V[0], kbar[0], ws),
                    lambda: store.seal(0, K[0].float(), V[0], kbar[0], ws), lambda: store.write(K[0], V[0], NP * P - 1, ws)):
            with pytest.raises(hsa.HsaError):
                bad()
    finally:
        store.close()


@pytest.mark.parametrize("use_store", [False, True])
@pytest.mark.parametrize("layout", [0, 1])
def test_step_over_quantised_pages(layout, use_store):
    """Rows are rotated, written and read as they are used together: queries and chunk keys rotated, history written as it
    is, selected pages read back rotated to their places, block selection, both branches and the merge on top -- against
    the oracle on the cache as it was read, and that cache against the quantised rows rotated in 64 bits."""
    H, d, Lq, P, NP, Kp, r = 2, 64, 256, 256, 8, 2, 64
    quant = hsa.make_quant(0, 64)
    Lc = Kp * P
    pairs = [16, 8, 8]
    inv = torch.cat([hsa.rope_freqs(2 * n)[0] for n in pairs]).cuda()
    rope = hsa.make_rope(inv, layout, pairs)
    at = torch.arange(Lc + Lq, device="cuda", dtype=torch.int32)
    grid = torch.stack([at // 64, at % 64 // 8, at % 8])
    pos_c, pos_q = grid[:, :Lc].contiguous(), grid[:, Lc:].contiguous()
    K, V = (to_dev(synth.normal_bf16((NP, P, H, d), 62, i)) for i in (1, 2))
    Q, Kq, Vq = (to_dev(synth.normal_bf16((Lq, H, d), 62, i)) for i in (3, 4, 5))
    E, F = (to_dev(synth.normal_bf16((r, Lc + Lq), 62, i, sigma=1 / math.sqrt(r))) for i in (6, 7))
    tau = torch.from_numpy(synth.tau_schedule(H).astype(np.float32)).cuda()
    z = torch.tensor([0.3, -0.4], device="cuda")
    store = pages = None
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    if use_store:
        store = QuantPageStore(quant, NP, 3, P, H, d)
        tables = store.page_tables()
        store.write(K.flatten(0, 1), V.flatten(0, 1), 0, ws)
    else:
        pages = Pages(hsa, quant, NP, P, H, d), Pages(hsa, quant, NP, P, H, d)
        tables = pages[0].table, pages[1].table
        hsa.hkv_quant_rows(quant, K.flatten(0, 1), V.flatten(0, 1), *tables, P, 0, ws)
    try:
        step = HkvHsaStep(H, d, Lq, P, NP, Kp, r, *tables, store=store, quant=quant, rope=rope, pos=pos_c)
        step.seal_pages(K)
        Qr, Kr = torch.empty_like(Q), torch.empty_like(Kq)
        hsa.hsa_rope(rope, pos_q, Q, Qr, Kq, Kr)
        out = step(Qr, Kr, Vq, tau, z, E, F).clone()
        torch.cuda.synchronize()
        assert hsa.hsa_status_read(step.ws) == 0 and hsa.hsa_status_read(ws) == 0
        sel = step.sel.cpu().tolist()
        kbar = step.kbar_pages.cpu().numpy()
        assert sel == sorted(oracle.select_pages(kbar, bits_of(Qr), Kp)[0].tolist())
        if use_store:
            assert all(store.residency()[0].cpu().numpy()[sel] >= 0)
        codes, scales = encode(K.float().cpu(), 0, 64)
        k = (codes.double().unflatten(-1, (-1, 64)) * scales.double()[..., None]).flatten(-2)[sel].flatten(0, 1)
        want, err = rope64(k, pos_c, inv, pairs, layout)
        err = err + 2.0 ** -23 * k.abs().amax()
        assert ((step.Kc.double().cpu() - want).abs() <= err + HALF_STEP[torch.bfloat16] * (want.abs() + err)).all()
        for j in range(Lc // 128):  # fp32 sums of 128 rows
            mean = step.kbar128[j].double().cpu()
            rows = want[128 * j:128 * (j + 1)]
            bound = (rows.abs().sum(0) * 130 * 2.0 ** -24 + err[128 * j:128 * (j + 1)].sum(0)) / 128
            assert ((mean - rows.mean(0)).abs() <= bound + 2.0 ** -24 * rows.mean(0).abs()).all()
        # blocks chosen from those means, both branches and the merge
        sb = step.selection
        gi = selection_lists(sb.inter_idx.cpu().numpy(), sb.inter_cnt.cpu().numpy())
        gq = selection_lists(sb.intra_idx.cpu().numpy(), sb.intra_cnt.cpu().numpy())
        p_inter = oracle.block_probs(oracle.block_means(bits_of(Qr), 128), step.kbar128.cpu().numpy().astype(np.float64), d ** -0.5)
        t = tau.cpu().numpy()
        keep = [[oracle.keep_blocks(p_inter[h, i], t[h]) for i in range(Lq // 128)] for h in range(H)]
        check_selection(gi, keep, p_inter, t, "inter")
        ref = oracle.block_select(bits_of(Qr), bits_of(step.Kc), bits_of(Kr), t)
        check_selection(gq, ref.intra, ref.p_intra, t, "intra")
        args = (bits_of(Qr), bits_of(step.Kc), bits_of(step.Vc), bits_of(Kr), bits_of(Vq), t, z.cpu().numpy(), bits_of(E), bits_of(F))
        assert_close(out.cpu().numpy(), oracle.hsa_step(*args, selection=oracle.Selection(gi, gq, None, None))["out"], "step")
        # the same through a prepared chunk's denoising step
        step.prepare_chunk(Qr, E, F)
        again = step.denoise_step(Qr, Kr, Vq, tau, z, E, F)
        assert_close(again.cpu().numpy(), out.cpu().numpy(), "denoising step")
        # a bf16 step over the rows as they were read gives the same selection and output
        plain = HkvHsaStep(H, d, Lq, P, Kp, Kp, r, *(torch.tensor([c[i * P:].data_ptr() for i in range(Kp)], device="cuda")
                                                     for c in (step.Kc, step.Vc)))
        plain.seal_pages(step.Kc.view(Kp, P, H, d))
        assert_close(plain(Qr, Kr, Vq, torch.ones_like(tau), z, E, F).cpu().numpy(),
                     step(Qr, Kr, Vq, torch.ones_like(tau), z, E, F).cpu().numpy(), "dense, bf16 pages")
    finally:
        if store is not None:
            store.close()


def test_step_retrieves_pages_by_the_queries_before_their_rotation():
    """A page whose keys point along the queries is found whatever the chunk's positions; queries that are half a turn
    further point the other way, and would retrieve the wrong pages."""
    quant, H, d, Lq, P, NP, Kp, r = hsa.make_quant(1, 64), 2, 64, 256, 256, 6, 2, 64
    inv = torch.full((d // 2,), math.pi / 8, dtype=torch.float64, device="cuda")
    rope = hsa.make_rope(inv, hsa.ROPE_HALF)
    toward = torch.from_numpy(np.sign(np.arange(d) % 3 - 0.5).astype(np.float32)).cuda().bfloat16()
    K = torch.stack([toward * (c + 0.5) for c in (-1, 0.5, 2, -2, 1, -3)])[:, None, None].expand(NP, P, H, d).contiguous()
    V = to_dev(synth.normal_bf16((NP, P, H, d), 63, 1))
    Q = (toward + 0.25 * to_dev(synth.normal_bf16((Lq, H, d), 63, 2))).bfloat16()
    Kq, Vq = (to_dev(synth.normal_bf16((Lq, H, d), 63, i)) for i in (3, 4))
    E, F = (to_dev(synth.normal_bf16((r, Kp * P + Lq), 63, i, sigma=1 / math.sqrt(r))) for i in (5, 6))
    tau, z = torch.full((H,), 0.9, device="cuda"), torch.zeros(H, device="cuda")
    pages = Pages(hsa, quant, NP, P, H, d), Pages(hsa, quant, NP, P, H, d)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    hsa.hkv_quant_rows(quant, K.flatten(0, 1), V.flatten(0, 1), pages[0].table, pages[1].table, P, 0, ws)
    pos_c, pos_q = (torch.full((n,), p, dtype=torch.int32, device="cuda") for n, p in ((Kp * P, 0), (Lq, 8)))
    step = HkvHsaStep(H, d, Lq, P, NP, Kp, r, pages[0].table, pages[1].table, quant=quant, rope=rope, pos=pos_c)
    step.seal_pages(K)
    Qr = torch.empty_like(Q)
    hsa.hsa_rope(rope, pos_q, Q, Qr)
    step(Qr, Kq, Vq, tau, z, E, F, q_pages=Q)
    assert step.sel.tolist() == [2, 4]
    step.prepare_chunk(Qr, E, F, q_pages=Q)
    assert step.sel.tolist() == [2, 4]
    step(Qr, Kq, Vq, tau, z, E, F)
    assert step.sel.tolist() == [3, 5]


def test_step_refuses_a_rotation_of_bf16_pages():
    inv = hsa.rope_freqs(64)[0].cuda()
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        HkvHsaStep(2, 64, 256, 256, 4, 2, 64, t, t, rope=hsa.make_rope(inv), pos=torch.zeros(512, dtype=torch.int32, device="cuda"))
