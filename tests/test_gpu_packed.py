"""GPU parity of the packed prefill (bifocal_prefill_packed) against the fp64 oracle, sequence by
sequence: lengths from 0 and 1 past several tiles, even, odd and single query-head groups, both
head sizes, both input types, both long-range forms, a window, dense and paged cache rows.

Every row that belongs to no sequence holds NaN in q, k and v, and every sequence's neighbours
are NaN in turn in one test: nothing of them may reach another sequence's result.

Tolerances: the output's are those of the other prefill tests (tests/gpu_helpers.py). A row's LSE
moves by at most the largest error of its scores; a score is a dot product of two operands rounded
to fp16 (2^-11 relative each), so it is off by at most scale * (2^-10 + 2^-20) * sum_d |q_d k_d|;
the bound taken is that, or 1e-3 where it is larger."""
import numpy as np
import pytest
import torch

import oracle.bifocal_ref as R
import rope_context_extension_bifocal_b200 as bfl
import seeded_inputs as si
from tests.gpu_helpers import MAX_ABS, REL_L2

pytestmark = pytest.mark.gpu
THETA = 1e6


def make(lens, hq, hkv, D, dtype, seed, lead=0, tail=0):
    """Packed inputs on the CPU, NaN before the first sequence and after the last."""
    g = si.generator(seed)
    T = lead + sum(lens) + tail
    x = [torch.randn(T, h, D, generator=g).to(dtype) for h in (hq, hkv, hkv)]
    for t in x:
        t[:lead] = float("nan")
        t[T - tail:] = float("nan")
    cu = torch.tensor([lead + sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)
    return x, cu


def lse_bound(q, k, w0, wp, mode):
    """[Hq, L] bound of a row's LSE error from the rounding of the rotated operands."""
    L, hq, D = q.shape
    g = hq // k.shape[1]
    G = R.dynamic_factor(L, wp)
    om = R.rope_omega(D, THETA)
    pos = np.arange(L, dtype=np.float64)
    far = pos / G if mode == si.FREQ_INTERP else np.floor(pos / G)
    out = np.zeros((hq, L))
    d = pos[:, None] - pos[None, :]
    for h in range(hq):
        b = []
        for p in (pos, far):
            qa = np.abs(R.rope_rotate(q[:, h], p, om))
            ka = np.abs(R.rope_rotate(k[:, h // g], p, om))
            b.append(qa @ ka.T)
        m = np.where(d < w0, b[0], b[1])
        m[d < 0] = 0
        out[h] = m.max(1) * (2.0 ** -10 + 2.0 ** -20) / np.sqrt(D)
    return np.maximum(out, 1e-3)


def check(lens, x, cu, out, lse, w0, wp, mode, window=False):
    q, k, v = (t.double().numpy() for t in x)
    for b, L in enumerate(lens):
        if L == 0:
            continue
        s = slice(int(cu[b]), int(cu[b + 1]))
        if window:
            ro, rl = R.sliding_window_attention(q[None, s], k[None, s], v[None, s], w0, THETA)
        else:
            ro, rl = R.bifocal_attention(q[None, s], k[None, s], v[None, s], w0, wp, THETA, mode)
        got, ref = out[s].cpu().double().numpy(), ro[0]
        d = got - ref
        assert np.abs(d).max() <= MAX_ABS and np.linalg.norm(d) <= REL_L2 * np.linalg.norm(ref), (b, L, np.abs(d).max())
        dl = np.abs(lse[:, s].cpu().double().numpy() - rl[0])
        assert np.all(dl <= lse_bound(q[s], k[s], w0, wp, mode)), (b, L, dl.max())


CASES = [
    # lens, hq, hkv, D, dtype, w0, w_pretrained, mode
    ([1], 2, 1, 128, torch.bfloat16, 4, 1, si.FREQ_INTERP),
    ([1, 0, 7, 129, 128, 1, 260], 8, 2, 128, torch.bfloat16, 60, 64, si.FREQ_INTERP),
    ([300, 33, 517], 4, 2, 128, torch.bfloat16, 128, 100, si.POS_ALIAS),
    ([700, 5], 8, 1, 128, torch.float32, 0, 128, si.FREQ_INTERP),
    ([140, 257, 2], 4, 2, 128, torch.bfloat16, 1, 50, si.POS_ALIAS),
    ([140, 257, 2], 6, 2, 128, torch.bfloat16, 100, 50, si.FREQ_INTERP),   # three heads a group: single-tile kernel
    ([385, 1, 0, 65], 3, 3, 128, torch.float32, 20, 40, si.POS_ALIAS),     # one head a group
    ([200, 63, 321], 6, 2, 64, torch.bfloat16, 50, 90, si.FREQ_INTERP),    # D = 64
    ([1, 129, 64], 4, 4, 64, torch.float32, 0, 30, si.POS_ALIAS),
    ([260, 100], 4, 2, 128, torch.bfloat16, 500, 1000, si.FREQ_INTERP),    # G = 1 throughout: the plain kernel
    ([260, 100, 300], 4, 2, 64, torch.bfloat16, 40, 280, si.FREQ_INTERP),  # G = 1 and 2 in one call
    ([260, 100, 300], 3, 1, 128, torch.bfloat16, 40, 280, si.POS_ALIAS),
    ([300, 63, 640], 8, 2, 64, torch.bfloat16, 130, 90, si.POS_ALIAS),     # D = 64, two heads a CTA
    ([1, 385], 5, 1, 64, torch.float32, 33, 100, si.FREQ_INTERP),          # D = 64, five heads a group
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_oracle(case):
    lens, hq, hkv, D, dtype, w0, wp, mode = CASES[case]
    x, cu = make(lens, hq, hkv, D, dtype, 900 + case, lead=3 * (case % 2), tail=5)
    dev = [t.cuda() for t in x]
    out, lse = bfl.bifocal_prefill_packed(*dev, cu.cuda(), max(lens), w0=w0, w_pretrained=wp, theta=THETA, mode=mode)
    assert bfl.last_device_error() == 0
    check(lens, x, cu, out, lse, w0, wp, mode)


@pytest.mark.parametrize("D", [64, 128])
def test_window(D):
    lens = [5, 300, 0, 129]
    x, cu = make(lens, 4, 2, D, torch.bfloat16, 77)
    out, lse = bfl.bifocal_prefill_packed(*(t.cuda() for t in x), cu.cuda(), 300, w0=40, w_pretrained=64, theta=THETA,
                                          flags=bfl.FLAG_WINDOW)
    assert bfl.last_device_error() == 0
    check(lens, x, cu, out, lse, 40, 64, si.FREQ_INTERP, window=True)


@pytest.mark.parametrize("hq,hkv,D", [(4, 2, 128), (3, 1, 128), (4, 2, 64), (3, 3, 64)])
def test_neighbours_do_not_leak(hq, hkv, D):
    """Sequences beside NaN and infinite ones give, bit for bit, what they give alone."""
    lens = [70, 200, 64, 129, 31]
    x, cu = make(lens, hq, hkv, D, torch.bfloat16, 5)
    kw = dict(w0=30, w_pretrained=50, theta=THETA)
    for keep in (1, 3):
        y = [t.clone() for t in x]
        for b in range(len(lens)):
            if b != keep:
                for t in y:
                    t[cu[b]:cu[b + 1]] = float("nan") if b % 2 else float("inf")
        out, lse = bfl.bifocal_prefill_packed(*(t.cuda() for t in y), cu.cuda(), 200, **kw)
        s = slice(int(cu[keep]), int(cu[keep + 1]))
        alone, alone_lse = bfl.bifocal_prefill_packed(*(t[s].contiguous().cuda() for t in x),
                                                      torch.tensor([0, lens[keep]], dtype=torch.int32).cuda(), 200, **kw)
        assert torch.equal(out[s], alone) and torch.equal(lse[:, s], alone_lse)
        bfl.last_device_error()  # the NaN sequences report fp16 operands out of range


@pytest.mark.parametrize("paged", [0, 1, 16, 48])
def test_cache_rows(paged):
    lens, hkv, D = [1, 130, 0, 77], 2, 128
    x, cu = make(lens, 4, hkv, D, torch.bfloat16, 31, tail=4)
    T = x[0].shape[0]
    if paged:
        need = [-(-n // paged) for n in lens]
        perm = torch.randperm(sum(need) + 2, generator=si.generator(3)).int()
        table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
        rows, nxt = (sum(need) + 2) * paged, 0
        for b, m in enumerate(need):
            table[b, :m] = perm[nxt:nxt + m]
            nxt += m
    else:
        table, rows = None, T + 9
    kc = torch.full((rows, hkv, D), 7.0, dtype=torch.bfloat16)
    vc, kpos = kc.clone(), torch.full((hkv, rows), -5, dtype=torch.int32)
    want_k, want_v, want_p = kc.clone(), vc.clone(), kpos.clone()
    for b, n in enumerate(lens):
        rot = R.rope_keys_for_cache(x[1][cu[b]:cu[b + 1]].double().numpy(), THETA)
        for j in range(n):
            r = int(table[b, j // paged]) * paged + j % paged if paged else int(cu[b]) + j
            want_k[r], want_v[r], want_p[:, r] = torch.from_numpy(rot[j]).bfloat16(), x[2][cu[b] + j], j
    dk, dv, dp = kc.cuda(), vc.cuda(), kpos.cuda()
    bfl.bifocal_prefill_packed(*(t.cuda() for t in x), cu.cuda(), 130, w0=40, w_pretrained=64, theta=THETA, kcache=dk,
                               vcache=dv, kpos=dp, page_size=paged, block_table=table.cuda() if paged else None)
    assert bfl.last_device_error() == 0
    assert torch.equal(dv.cpu(), want_v) and torch.equal(dp.cpu(), want_p)
    # keys: within one bf16 step of the fp64 rotation (half a step, and fp32 arithmetic at a rounding border)
    assert torch.all((dk.cpu().double() - want_k.double()).abs() <= want_k.double().abs() * 2.0 ** -7 + 1e-5)


def test_rows_of_no_sequence_are_left():
    lens = [40, 60]
    x, cu = make(lens, 4, 2, 128, torch.bfloat16, 8, lead=7, tail=130)
    out = torch.full((237, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    bfl.bifocal_prefill_packed(*(t.cuda() for t in x), cu.cuda(), 60, w0=40, w_pretrained=64, theta=THETA, out=out)
    assert bfl.last_device_error() == 0
    assert torch.all(out[:7] == 3) and torch.all(out[107:] == 3)


def test_equals_the_equal_length_prefill():
    """Equal lengths: the packed call's rows are those of bifocal_prefill, bit for bit."""
    g = si.generator(12)
    q, k, v = (torch.randn(3, 200, h, 128, generator=g).bfloat16().cuda() for h in (4, 2, 2))
    kw = dict(w0=50, w_pretrained=60, theta=THETA)
    want, want_lse, _, _ = bfl.bifocal_prefill(q, k, v, **kw)
    cu = torch.tensor([0, 200, 400, 600], dtype=torch.int32).cuda()
    out, lse = bfl.bifocal_prefill_packed(*(t.view(600, -1, 128) for t in (q, k, v)), cu, 200, **kw)
    assert torch.equal(out.view_as(want), want)
    assert torch.equal(lse.view(4, 3, 200).transpose(0, 1), want_lse)


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [0, 50, 101], [-1, 100], [0, 90, 100]])
def test_bad_boundaries_are_reported(cu):
    x, _ = make([100], 4, 2, 128, torch.bfloat16, 8)
    out = torch.full((100, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    bfl.bifocal_prefill_packed(*(t.cuda() for t in x), torch.tensor(cu, dtype=torch.int32).cuda(), 80, w0=40,
                               w_pretrained=64, theta=THETA, out=out)
    assert bfl.last_device_error() == bfl.STATUS_INDEX
    assert torch.all(out == 3)


def test_bad_page_is_reported():
    x, cu = make([100], 4, 2, 128, torch.bfloat16, 8)
    table = torch.tensor([[0, 9, 1, -3]], dtype=torch.int32).cuda()
    kc = torch.full((4 * 32, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    out, lse = bfl.bifocal_prefill_packed(*(t.cuda() for t in x), cu.cuda(), 100, w0=40, w_pretrained=64, theta=THETA,
                                          kcache=kc, vcache=vc, page_size=32, block_table=table)
    assert bfl.last_device_error() == bfl.STATUS_INDEX
    assert torch.all(vc[64:] == 7) and torch.equal(vc[:32], x[2][:32].cuda()) and torch.equal(vc[32:64], x[2][64:96].cuda())
    check([100], x, cu, out, lse, 40, 64, si.FREQ_INTERP)


@pytest.mark.parametrize("fill", [0x00, 0xff])
@pytest.mark.parametrize("hq,hkv,D,window,w0,wp", [(4, 2, 128, False, 128, 512), (4, 2, 64, False, 128, 512), (3, 1, 128, False, 128, 512),
                                                   (4, 2, 128, True, 300, 512), (8, 2, 128, False, 700, 900)])
def test_rows_past_a_sequence_change_no_bit(hq, hkv, D, window, w0, wp, fill):
    """The last query tile of a sequence of nine tiles and several unmasked ones holds rows of the next sequence: of one
    without long-range forms (whatever the workspace held there: zeros, or NaN), of one whose scores outgrow any
    reference. The results are those of the sequence alone, and of bifocal_prefill where it has the same kernel, bit for bit."""
    lens = [1100, 200, 1061, 600]
    x, cu = make(lens, hq, hkv, D, torch.bfloat16, 15)
    x[0][cu[3]:] *= 64
    kw = dict(w0=w0, w_pretrained=wp, theta=THETA, flags=bfl.FLAG_WINDOW if window else 0)
    p = bfl.make_params(hq, hkv, D, w0, wp, THETA)
    ws = torch.full((bfl.prefill_packed_workspace_size(bfl.DTYPE_BF16, 4, sum(lens), p),), fill, dtype=torch.uint8, device="cuda")
    out, lse = bfl.bifocal_prefill_packed(*(t.cuda() for t in x), cu.cuda(), 1100, workspace=ws, **kw)
    assert bfl.last_device_error() == 0
    for b in (0, 2):
        s = slice(int(cu[b]), int(cu[b + 1]))
        one = [t[s].contiguous().cuda() for t in x]
        alone, alone_lse = bfl.bifocal_prefill_packed(*one, torch.tensor([0, lens[b]], dtype=torch.int32).cuda(), 1100, **kw)
        assert torch.equal(out[s], alone) and torch.equal(lse[:, s], alone_lse), b
        if D == 128:
            dense, dense_lse, _, _ = bfl.bifocal_prefill(*(t[None] for t in one), **kw)
            assert torch.equal(out[s], dense[0]) and torch.equal(lse[:, s], dense_lse[0]), b
