"""The operators together, as a server runs them: packed prompts fill a paged cache, the keys' weights are taken,
the cache is cut in place, decoding goes on over the kept slots, and a step that outgrows the budget evicts again.
Every step is checked against the fp64 references fed with the state the GPU holds before it."""
import numpy as np
import pytest
import torch

import oracle.bifocal_ref as R
import rope_context_extension_bifocal_b200 as bfl
import seeded_inputs as si
from tests.kept_ref import THETA, choose, decode_kept, moves, page_table, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,D,mode", [(8, 2, 128, si.FREQ_INTERP), (6, 2, 64, si.POS_ALIAS)])
def test_prompt_weights_evict_decode_evict(hq, hkv, D, mode):
    lens, page, budget, recent, sink, obs = [400, 90, 211], 16, 128, 32, 4, 48
    g, T, B = si.generator(11), sum(lens), len(lens)
    rope = dict(w0=60, w_pretrained=100, theta=THETA, mode=mode)
    table, pages = page_table([n + 16 for n in lens], page, g)
    q, k, v = (torch.randn(T, h, D, generator=g).bfloat16() for h in (hq, hkv, hkv))
    cu = torch.tensor([0, 400, 490, 701], dtype=torch.int32).cuda()
    rows = pages * page
    kc = torch.full((rows, hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc, kpos = kc.clone(), torch.full((hkv, rows), -1, dtype=torch.int32, device="cuda")
    kw = torch.full((hkv, rows), float("nan"), device="cuda")
    t = table.cuda()
    out, lse = bfl.bifocal_prefill_packed(q.cuda(), k.cuda(), v.cuda(), cu, 400, kcache=kc, vcache=vc, kpos=kpos, page_size=page,
                                          block_table=t, **rope)
    bfl.bifocal_key_weights(q.cuda(), k.cuda(), lse, cu, 400, obs, kweight=kw, page_size=page, block_table=t, **rope)
    seq, now = torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor([n - 1 for n in lens], dtype=torch.int32).cuda()
    for b, n in enumerate(lens):
        r = rows_of(table, page, b, n)
        s = slice(int(cu[b]), int(cu[b + 1]))
        ro, _ = R.bifocal_attention(q[None, s].double().numpy(), k[None, s].double().numpy(), v[None, s].double().numpy(),
                                    60, 100, THETA, mode)
        assert np.linalg.norm(out[s].cpu().double().numpy() - ro[0]) <= 5e-3 * np.linalg.norm(ro[0])
        # every query of the window gives its group's heads a total of one each
        total = kw[:, r].double().sum(1).cpu().numpy()
        assert np.allclose(total, hq // hkv * min(n, obs), rtol=1e-3)

    def evict():
        before = [x.cpu() for x in (kc, vc, kpos, kw)]
        held, at = seq.tolist(), now.tolist()
        bfl.bifocal_cache_evict(kc, vc, kpos, kw, page, t, seq, now, 416, budget, recent=recent, sink=sink, new_lens=seq)
        assert bfl.last_device_error() == 0 and seq.tolist() == [min(n, budget) for n in held]
        want = [x.clone() for x in before]
        for b, n in enumerate(held):
            r = rows_of(table, page, b, n)
            for h in range(hkv):
                kept = choose(before[2][h, r].tolist(), before[3][h, r].tolist(), at[b], min(n, budget), recent, sink)
                for f, to in moves(kept, n, True):
                    for i, x in enumerate(want):
                        if i < 2:
                            x[r[to], h] = before[i][r[f], h]
                        else:
                            x[h, r[to]] = before[i][h, r[f]]
        for x, y in zip((kc, vc, kpos, kw), want):
            bits = torch.int16 if x.dtype == torch.bfloat16 else torch.int32
            assert torch.equal(x.cpu().view(bits), y.view(bits))

    evict()
    for step in range(5):
        seq += 1
        now += 1
        q1, k1, v1 = (torch.randn(B, h, D, generator=g).bfloat16() for h in (hq, hkv, hkv))
        before = kw.cpu()
        out, lse = bfl.bifocal_decode_kept(q1.cuda(), k1.cuda(), v1.cuda(), kc, vc, kpos, kw, page, t, seq, now, 416, **rope)
        assert bfl.last_device_error() == 0
        for b, n in enumerate(seq.tolist()):
            r = rows_of(table, page, b, n)
            for h in range(hkv):
                hs = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                ro, rl, w, _ = decode_kept(q1[b, hs].double().numpy(), kc[r, h].cpu().double().numpy(),
                                           vc[r, h].cpu().double().numpy(), kpos[h, r].cpu().numpy(), int(now[b]), 60, 100, mode)
                assert np.abs(lse[b, hs].cpu().numpy() - rl).max() <= 1e-4
                assert np.linalg.norm(out[b, hs].cpu().double().numpy() - ro) <= 5e-3 * np.linalg.norm(ro)
                old = before[h, r].double().numpy()
                old[-1] = 0
                assert np.abs(kw[h, r].cpu().double().numpy() - old - w).max() <= 1e-4
        if step % 2:
            evict()
