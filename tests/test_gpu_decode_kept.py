"""bifocal_decode_kept against the fp64 reference, head by head: every group size, both head sizes and
long-range forms, positions in any order and far out, one slot to many ranges of slots, pages of any size.
Every pool row that holds no slot is NaN, and so are the positions' and weights' other places.

Tolerances. Scores are formed in fp32 from operands turned by angles within 2^-23 turns and sines within
2^-21; per score that is at most EPS = 4e-6 of scale |q| |k| (2 pi 2^-23 + 2^-21 on the key, half of that on the
query, and the fp32 sums). With d the largest such error of a row, its probabilities are off by 2 d + 2e-6
relative, its LSE by d + 1e-6 (1 + |lse|), its output by that share of sum p |v| and half a bf16 step, and a
weight, summed over a group, by that share of itself and half an fp32 step of what it is added to."""
import numpy as np
import pytest
import torch

import oracle.bifocal_ref as R
import rope_context_extension_bifocal_b200 as bfl
import seeded_inputs as si
from tests.kept_ref import THETA, decode_kept, page_table, rotate, rows_of

pytestmark = pytest.mark.gpu
EPS = 4e-6


def make(lens, hq, hkv, D, page, seed, stretch=4, start=0, order="random"):
    g = si.generator(seed)
    B = len(lens)
    table, pages = page_table(lens, page, g)
    rows = pages * page
    s = dict(table=table, page=page, lens=lens, max_len=max(lens))
    s["kc"] = torch.full((rows, hkv, D), float("nan"), dtype=torch.bfloat16)
    s["vc"] = s["kc"].clone()
    s["kpos"] = torch.full((hkv, rows), -(1 << 30), dtype=torch.int32)
    s["kw"] = torch.full((hkv, rows), float("nan"))
    now = []
    for b, n in enumerate(lens):
        r = rows_of(table, page, b, n)
        now.append(start + stretch * n)
        for h in range(hkv):
            pos = start + torch.randperm(stretch * n, generator=g)[:n - 1]
            if order == "sorted":
                pos = pos.sort()[0]
            s["kpos"][h, r[:-1]] = pos.int()
            s["kc"][r[:-1], h] = torch.randn(n - 1, D, generator=g).bfloat16()
            s["vc"][r[:-1], h] = torch.randn(n - 1, D, generator=g).bfloat16()
            s["kw"][h, r[:-1]] = torch.rand(n - 1, generator=g) * 3
    s["now"] = torch.tensor(now, dtype=torch.int32)
    s["q"], s["kn"], s["vn"] = (torch.randn(B, h, D, generator=g).bfloat16() for h in (hq, hkv, hkv))
    return s


def call(s, dev=None, **kw):
    d = dev or {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in s.items()}
    if "len_t" not in d:
        d["len_t"] = torch.tensor(s["lens"], dtype=torch.int32).cuda()
    out, lse = bfl.bifocal_decode_kept(d["q"], d["kn"], d["vn"], d["kc"], d["vc"], d["kpos"], d["kw"], s["page"], d["table"],
                                       d["len_t"], d["now"], s["max_len"], theta=THETA, **kw)
    return d, out, lse


def check(s, d, out, lse, w0, wp, mode, window=False, steps=1):
    out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    kc, vc, kpos, kw = (d[x].cpu() for x in ("kc", "vc", "kpos", "kw"))
    B, hq, D = s["q"].shape
    hkv = s["kn"].shape[1]
    g = hq // hkv
    touched = torch.zeros(kc.shape[0], dtype=torch.bool)
    for b, n in enumerate(s["lens"]):
        r = rows_of(s["table"], s["page"], b, n)
        touched[r] = True
        now, last = int(s["now"][b]), r[-1]
        assert torch.equal(vc[last], s["vn"][b]) and torch.all(kpos[:, last] == now)
        want = rotate(s["kn"][b].double().numpy(), np.full(hkv, float(now)))
        assert np.all(np.abs(kc[last].double().numpy() - want) <= np.abs(want) * 2.0 ** -7 + 1e-5)
        assert torch.equal(kc[r[:-1]], s["kc"][r[:-1]]) and torch.equal(kpos[:, r[:-1]], s["kpos"][:, r[:-1]])
        for h in range(hkv):
            q = s["q"][b, h * g:(h + 1) * g].double().numpy()
            keys, vals = kc[r, h].double().numpy(), vc[r, h].double().numpy()
            ro, rl, w, pv = decode_kept(q, keys, vals, kpos[h, r].numpy(), now, w0, wp, mode, window)
            dlt = EPS / np.sqrt(D) * np.linalg.norm(q, axis=1) * np.linalg.norm(keys, axis=1).max()
            rel = (2 * dlt + 2e-6)[:, None]
            assert np.all(np.abs(out[b, h * g:(h + 1) * g] - ro) <= 2.0 ** -8 * np.abs(ro) + rel * pv + 1e-30), (b, h)
            assert np.all(np.abs(lse[b, h * g:(h + 1) * g] - rl) <= dlt + 1e-6 * (1 + np.abs(rl))), (b, h)
            if s["kw"] is not None and d["kw"] is not None:
                old = s["kw"][h, r].double().numpy()
                old[-1] = 0  # the new token's slot starts at zero, whatever it held
                got = kw[h, r].double().numpy()
                assert np.all(np.abs(got - old - w) <= rel.max() * w + 2.0 ** -23 * (old + w)), (b, h)
    rest = ~touched
    assert torch.isnan(kc[rest].float()).all() and torch.isnan(kw[:, rest]).all()


CASES = [
    # lens, hq, hkv, D, page, w0, w_pretrained, mode, stretch, order
    ([1], 1, 1, 128, 16, 4, 1, si.FREQ_INTERP, 1, "sorted"),
    ([1, 2, 9, 65, 700], 8, 2, 128, 16, 100, 64, si.FREQ_INTERP, 4, "random"),
    ([130, 64, 63], 6, 2, 128, 48, 20, 100, si.POS_ALIAS, 4, "random"),
    ([200, 17], 10, 2, 128, 1, 0, 50, si.POS_ALIAS, 2, "sorted"),
    ([333, 5], 16, 2, 128, 64, 200, 100, si.FREQ_INTERP, 8, "random"),
    ([150], 2, 2, 128, 16, 1, 30, si.FREQ_INTERP, 3, "random"),
    ([150, 31], 4, 2, 64, 16, 60, 30, si.POS_ALIAS, 3, "random"),
    ([2050, 40], 4, 1, 64, 128, 300, 500, si.FREQ_INTERP, 4, "sorted"),
    ([77], 8, 1, 64, 7, 0, 20, si.FREQ_INTERP, 4, "random"),
    ([90, 8], 3, 3, 64, 16, 9, 20, si.POS_ALIAS, 4, "random"),
    ([300], 8, 2, 128, 16, 50, 100000, si.FREQ_INTERP, 4, "random"),     # G = 1: nothing is turned
    ([300], 8, 2, 128, 16, 100000, 100, si.FREQ_INTERP, 4, "random"),    # everything is local
    ([5000, 3], 4, 1, 128, 32, 700, 3000, si.FREQ_INTERP, 3, "sorted"),  # several ranges
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_reference(case):
    lens, hq, hkv, D, page, w0, wp, mode, stretch, order = CASES[case]
    s = make(lens, hq, hkv, D, page, 200 + case, stretch, 0, order)
    d, out, lse = call(s, w0=w0, w_pretrained=wp, mode=mode)
    assert bfl.last_device_error() == 0
    check(s, d, out, lse, w0, wp, mode)


@pytest.mark.parametrize("mode", [si.FREQ_INTERP, si.POS_ALIAS])
@pytest.mark.parametrize("start", [130000, 1 << 20, 1 << 30])
def test_far_positions(start, mode):
    """The reduced angle stays exact far out (the fp64 reference's own angle is exact to 2^30 2^-52)."""
    s = make([120, 33], 4, 2, 128, 16, 17, 64, start)
    d, out, lse = call(s, w0=500, w_pretrained=32768, mode=mode)
    assert bfl.last_device_error() == 0
    check(s, d, out, lse, 500, 32768, mode)


def test_window_and_rows_it_empties():
    s = make([100, 64, 1], 4, 2, 128, 16, 18, 4)
    d, out, lse = call(s, w0=30, w_pretrained=64, flags=bfl.FLAG_WINDOW)
    assert bfl.last_device_error() == 0
    check(s, d, out, lse, 30, 64, si.FREQ_INTERP, window=True)
    d, out, lse = call(s, w0=1, w_pretrained=64, flags=bfl.FLAG_WINDOW)  # the new token alone is left
    check(s, d, out, lse, 1, 64, si.FREQ_INTERP, window=True)
    assert torch.equal(out.cpu().view(3, 2, 2, 128), s["vn"][:, :, None].expand(3, 2, 2, 128))


def test_without_weights_nothing_else_changes():
    s = make([200, 3], 4, 2, 128, 16, 19)
    kw = dict(w0=50, w_pretrained=64)
    d, out, lse = call(s, **kw)
    e = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in s.items()}
    e["kw"] = None
    e, out2, lse2 = call(s, e, **kw)
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(d["kpos"], e["kpos"])
    assert torch.equal(d["vc"].view(torch.int16), e["vc"].view(torch.int16))


def test_equals_the_paged_decode_where_slots_are_positions():
    """Slots in order of their positions: the same step as bifocal_decode_paged (whose operands are fp16)."""
    s = make([500, 40], 8, 2, 128, 16, 20, 1, 0, "sorted")
    for b, n in enumerate(s["lens"]):
        r = rows_of(s["table"], 16, b, n)
        s["kpos"][:, r] = torch.arange(n, dtype=torch.int32)
    s["now"] = torch.tensor(s["lens"], dtype=torch.int32) - 1
    kw = dict(w0=50, w_pretrained=64)
    kc, vc = s["kc"].cuda(), s["vc"].cuda()
    d, out, lse = call(s, **kw)
    table = s["table"].clamp(min=0).cuda()
    ref, ref_lse = bfl.bifocal_decode_paged(s["q"].cuda(), s["kn"].cuda(), s["vn"].cuda(), kc, vc, 16, table,
                                            d["len_t"], 500, theta=THETA, **kw)
    assert torch.equal(kc.view(torch.int16), d["kc"].view(torch.int16)) and torch.equal(vc.view(torch.int16), d["vc"].view(torch.int16))
    assert (lse - ref_lse).abs().max() <= 2e-3 and (out.float() - ref.float()).norm() <= 1e-2 * ref.float().norm()


def test_bad_lengths_positions_and_pages_are_reported():
    s = make([60, 50, 40], 4, 2, 128, 16, 21)
    good = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in s.items()}
    for lens, now in (([61, 50, 0], None), (None, [-1, int(s["now"][1]), 0x7fffffff])):
        d = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in good.items()}
        if lens:
            d["len_t"] = torch.tensor(lens, dtype=torch.int32).cuda()
        if now:
            d["now"] = torch.tensor(now, dtype=torch.int32).cuda()
        d, out, lse = call(s, d, w0=20, w_pretrained=64)
        assert bfl.last_device_error() == bfl.STATUS_INDEX
        assert torch.isnan(out[[0, 2]].float()).all() and torch.isnan(lse[[0, 2]]).all() and not torch.isnan(out[1].float()).any()
        r = np.concatenate([rows_of(s["table"], 16, b, s["lens"][b]) for b in (0, 2)])
        assert torch.equal(d["kpos"][:, r].cpu(), s["kpos"][:, r]) and torch.isnan(d["kc"][r[59]].float()).all()
    d = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in good.items()}
    d["table"][0, 3], d["table"][2, 1] = 999, -1  # sequence 0's last page, one in the middle of sequence 2
    before = {k: d[k].clone() for k in ("kc", "vc", "kpos", "kw")}
    d, out, lse = call(s, d, w0=20, w_pretrained=64)
    assert bfl.last_device_error() == bfl.STATUS_INDEX
    assert not torch.isnan(out.float()).any()
    r = rows_of(s["table"], 16, 0, 60)[48:]
    assert torch.equal(d["kpos"][:, r], before["kpos"][:, r]) and torch.equal(d["kc"][r].view(torch.int16), before["kc"][r].view(torch.int16))


def test_captured_replayed_and_on_another_stream():
    s = make([300, 20], 8, 2, 128, 16, 22)
    kw = dict(w0=50, w_pretrained=64)
    want, out0, lse0 = call(s, **kw)
    d = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in s.items()}
    d["len_t"] = torch.tensor(s["lens"], dtype=torch.int32).cuda()
    p = bfl.make_params(8, 2, 128, 50, 64, THETA)
    ws = torch.empty(bfl.decode_kept_workspace_size(2, 300, True, p), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        d, out, lse = call(s, d, workspace=ws, **kw)
    for _ in range(2):
        d["kw"].copy_(s["kw"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, out0) and torch.equal(lse, lse0)
        assert torch.equal(d["kw"].view(torch.int32), want["kw"].view(torch.int32))
    d["kw"].copy_(s["kw"])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        d, out, lse = call(s, d, **kw)
    side.synchronize()
    assert torch.equal(out, out0) and torch.equal(d["kw"].view(torch.int32), want["kw"].view(torch.int32))


def test_position_zero_is_not_turned():
    """The key of position 0 turned by the angle of position 0, and a query whose long-range angle is 0 (position 1, G = 2,
    position aliasing): products of x with y halves alone, so the score is 0 whatever its operands' size. The new key is
    0 as well: both probabilities are 1/2, the log-sum-exp is log 2."""
    page, D, hkv, hq = 16, 128, 2, 8
    kc, vc = torch.zeros(16, hkv, D, dtype=torch.bfloat16), torch.zeros(16, hkv, D, dtype=torch.bfloat16)
    kc[0, :, :64], vc[0] = 256, 3
    q, kn = torch.zeros(1, hq, D, dtype=torch.bfloat16), torch.zeros(1, hkv, D, dtype=torch.bfloat16)
    q[..., 64:] = 256
    kpos, kw = torch.zeros(hkv, 16, dtype=torch.int32).cuda(), torch.zeros(hkv, 16).cuda()
    one = torch.tensor([1], dtype=torch.int32).cuda()
    out, lse = bfl.bifocal_decode_kept(q.cuda(), kn.cuda(), kn.cuda(), kc.cuda(), vc.cuda(), kpos, kw, page,
                                       torch.zeros(1, 1, dtype=torch.int32).cuda(), one + 1, one, 2, w0=1, w_pretrained=1,
                                       theta=THETA, mode=si.POS_ALIAS)
    assert bfl.last_device_error() == 0
    assert (lse - np.log(2)).abs().max() <= 1e-6 * (1 + np.log(2))
    assert (kw[:, :2] - hq / hkv / 2).abs().max() <= 2e-6 * hq / hkv / 2 and torch.all(out == 1.5)


def test_keys_and_values_of_a_bad_page_read_as_zeros():
    """The page of the new token's slot, and one in the middle: the results are those of zero keys and values there (a
    score of 0, whatever the position), the new token's among them, and nothing of these slots is written."""
    s = make([60, 50, 40], 4, 2, 128, 16, 21)
    kw = dict(w0=20, w_pretrained=64)
    d = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in s.items()}
    bad = {0: slice(48, 60), 1: slice(0, 0), 2: slice(16, 32)}
    d["table"] = d["table"].clone()
    d["table"][0, 3], d["table"][2, 1] = 999, -1
    d, out, lse = call(s, d, **kw)
    assert bfl.last_device_error() == bfl.STATUS_INDEX
    out, lse, weight = (t.cpu().double().numpy() for t in (out, lse, d["kw"]))
    for b, n in enumerate(s["lens"]):
        r = rows_of(s["table"], 16, b, n)
        now = int(s["now"][b])
        good = np.ones(n, dtype=bool)
        good[bad[b]] = False
        for h in range(2):
            q = s["q"][b, 2 * h:2 * h + 2].double().numpy()
            keys, vals = d["kc"].cpu()[r, h].double().numpy(), d["vc"].cpu()[r, h].double().numpy()
            keys[~good], vals[~good] = 0, 0
            pos = d["kpos"].cpu()[h, r].numpy().copy()
            pos[~good] = 0
            ro, rl, w, pv = decode_kept(q, keys, vals, pos, now, 20, 64, si.FREQ_INTERP)
            dlt = EPS / np.sqrt(128) * np.linalg.norm(q, axis=1) * np.linalg.norm(keys, axis=1).max()
            rel = (2 * dlt + 2e-6)[:, None]
            assert np.all(np.abs(out[b, 2 * h:2 * h + 2] - ro) <= 2.0 ** -8 * np.abs(ro) + rel * pv + 1e-30), (b, h)
            assert np.all(np.abs(lse[b, 2 * h:2 * h + 2] - rl) <= dlt + 1e-6 * (1 + np.abs(rl))), (b, h)
            old = s["kw"][h, r].double().numpy()
            old[-1] = 0
            err = np.abs(weight[h, r] - old - w)[good]
            assert np.all(err <= (rel.max() * w + 2.0 ** -23 * (old + w))[good]), (b, h)
            same = d["kw"].cpu()[h, r[~good]].view(torch.int32), s["kw"][h, r[~good]].view(torch.int32)
            assert torch.equal(*same) and torch.equal(d["kpos"].cpu()[h, r[~good]], s["kpos"][h, r[~good]])
        assert torch.equal(d["kc"].cpu()[r[~good]].view(torch.int16), s["kc"][r[~good]].view(torch.int16))
        assert torch.equal(d["vc"].cpu()[r[~good]].view(torch.int16), s["vc"][r[~good]].view(torch.int16))
