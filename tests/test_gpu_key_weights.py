"""bifocal_key_weights against the fp64 definition: lengths from one token over several tiles, windows of one
query to all of them, every group size, both head sizes, input types and long-range forms, dense and paged
destinations. Log-sum-exps that no weight asks for are NaN, and so are rows of no sequence.

Tolerance. A score is off by at most EPS = 4e-6 of scale |q| |k|: operands split in two fp16 parts (3 2^-22 of
sum |q_d k_d|), fp32 rotations (2^-21) and fp32 sums on the tensor cores. The log-sum-exp enters in fp32 (2^-23 of
it, up to 1e-6 here) and ex2 adds 2^-22. So each term, and their sum, is off by that share of itself."""
import math

import numpy as np
import pytest
import torch

import oracle.bifocal_ref as R
import rope_context_extension_bifocal_b200 as bfl
import seeded_inputs as si
from tests.kept_ref import THETA, far, page_table, rotate, rows_of

pytestmark = pytest.mark.gpu
EPS = 4e-6


def scores(q, k, w0, wp, mode, window):
    """[Hq, L, L] scores of one sequence, -inf where masked, and the largest scale |q| |k|."""
    L, hq, D = q.shape
    g = hq // k.shape[1]
    G = R.dynamic_factor(L, wp)
    pos = np.arange(L, dtype=np.float64)
    d = pos[:, None] - pos[None, :]
    out = np.empty((hq, L, L))
    for h in range(hq):
        a = rotate(q[:, h], pos) @ rotate(k[:, h // g], pos).T
        b = rotate(q[:, h], far(pos, G, mode)) @ rotate(k[:, h // g], far(pos, G, mode)).T
        out[h] = np.where(d < w0, a, -np.inf if window else b) / math.sqrt(D)
        out[h][d < 0] = -np.inf
    size = np.linalg.norm(q, axis=2).max() * np.linalg.norm(k, axis=2).max() / math.sqrt(D)
    return out, size


def run(lens, hq, hkv, D, dtype, obs, w0, wp, mode, seed, page=None, window=False, lead=0, tail=3):
    g = si.generator(seed)
    T = lead + sum(lens) + tail
    q, k = (torch.randn(T, h, D, generator=g).to(dtype) for h in (hq, hkv))
    cu = [lead + sum(lens[:i]) for i in range(len(lens) + 1)]
    lse = torch.full((hq, T), float("nan"))
    want, size = [], 1.0
    for b, n in enumerate(lens):
        s = slice(cu[b], cu[b] + n)
        if n == 0:
            want.append(np.zeros((hkv, 0)))
            continue
        x, sz = scores(q[s].double().numpy(), k[s].double().numpy(), w0, wp, mode, window)
        size = max(size, sz)
        m = x.max(2)
        l = (m + np.log(np.exp(x - m[..., None]).sum(2))).astype(np.float32)
        lo = max(0, n - obs)
        lse[:, cu[b] + lo:cu[b] + n] = torch.from_numpy(l[:, lo:])
        p = np.exp(x[:, lo:] - l[:, lo:, None].astype(np.float64)).sum(1)
        want.append(p.reshape(hkv, hq // hkv, n).sum(1))
    for t in (q, k):
        t[:lead] = float("nan")
        t[T - tail:] = float("nan")
    table, rows = None, T
    if page:
        table, pages = page_table(lens, page, g)
        rows = pages * page
    kw = torch.full((hkv, rows), -3.0, device="cuda")
    got = bfl.bifocal_key_weights(q.cuda(), k.cuda(), lse.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), max(lens), obs,
                                  w0=w0, w_pretrained=wp, theta=THETA, mode=mode, kweight=kw, page_size=page or 0,
                                  block_table=None if table is None else table.cuda(),
                                  flags=bfl.FLAG_WINDOW if window else 0)
    assert got is kw and bfl.last_device_error() == 0
    kw = kw.cpu().double().numpy()
    left = np.ones(rows, dtype=bool)
    tol = EPS * size + 4e-6
    for b, n in enumerate(lens):
        at = rows_of(table, page, b, n) if page else np.arange(cu[b], cu[b] + n)
        left[at] = False
        err = np.abs(kw[:, at] - want[b])
        assert np.all(err <= tol * want[b] + 1e-30), (b, n, (err / np.maximum(want[b], 1e-30)).max(), tol)
    assert np.all(kw[:, left] == -3.0)


CASES = [
    # lens, hq, hkv, D, dtype, obs, w0, w_pretrained, mode, page
    ([1], 1, 1, 128, torch.bfloat16, 1, 4, 1, si.FREQ_INTERP, None),
    ([1, 0, 7, 129, 300], 8, 2, 128, torch.bfloat16, 64, 60, 64, si.FREQ_INTERP, 16),
    ([513, 33], 4, 2, 128, torch.bfloat16, 10 ** 6, 128, 100, si.POS_ALIAS, None),
    ([300, 5], 6, 2, 128, torch.float32, 100, 0, 50, si.FREQ_INTERP, 48),
    ([257, 128], 3, 3, 128, torch.bfloat16, 1, 1, 50, si.POS_ALIAS, None),
    ([700], 8, 1, 128, torch.bfloat16, 200, 300, 200, si.FREQ_INTERP, 1),
    ([400, 90], 10, 2, 64, torch.bfloat16, 10 ** 6, 130, 100, si.FREQ_INTERP, 16),
    ([400, 1, 90], 4, 4, 64, torch.float32, 37, 60, 100, si.POS_ALIAS, None),
    ([260, 100], 4, 2, 128, torch.bfloat16, 10 ** 6, 500, 1000, si.FREQ_INTERP, None),  # G = 1
    ([260, 100, 300], 4, 2, 128, torch.bfloat16, 130, 40, 280, si.POS_ALIAS, None),     # G = 1 and 2 in one call
    ([1400], 2, 1, 128, torch.bfloat16, 10 ** 6, 513, 300, si.FREQ_INTERP, None),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_definition(case):
    lens, hq, hkv, D, dtype, obs, w0, wp, mode, page = CASES[case]
    run(lens, hq, hkv, D, dtype, obs, w0, wp, mode, 600 + case, page, lead=5 * (case % 2))


@pytest.mark.parametrize("D", [64, 128])
def test_window(D):
    run([300, 20], 4, 2, D, torch.bfloat16, 100, 40, 64, si.FREQ_INTERP, 50, window=True)


def test_neighbours_and_earlier_queries_do_not_leak():
    """NaN and infinite neighbours, and NaN queries before the window, change nothing, bit for bit."""
    g = si.generator(9)
    lens = [70, 200, 64]
    q, k = torch.randn(334, 4, 128, generator=g).bfloat16(), torch.randn(334, 2, 128, generator=g).bfloat16()
    lse = torch.rand(4, 334, generator=g) + 4
    cu = torch.tensor([0, 70, 270, 334], dtype=torch.int32).cuda()
    kw = dict(w0=30, w_pretrained=50, theta=THETA)
    want = bfl.bifocal_key_weights(q.cuda(), k.cuda(), lse.cuda(), cu, 200, 50, **kw)
    assert bfl.last_device_error() == 0
    q[:70], k[:70], lse[:, :70] = float("nan"), float("inf"), float("nan")
    q[270:], k[270:], lse[:, 270:] = float("inf"), float("nan"), float("-inf")
    q[70:220], lse[:, 70:220] = float("nan"), float("nan")
    got = bfl.bifocal_key_weights(q.cuda(), k.cuda(), lse.cuda(), cu, 200, 50, **kw)
    assert torch.equal(got[:, 70:270], want[:, 70:270])
    bfl.last_device_error()


def test_many_queries():
    """From 16384 (query, head) rows on the queries are single fp16 values. Rounding element d moves it by at most
    2^-11 of itself, evenly spread: 2^-11 / sqrt(3) in the root mean square. A score is then off by a standard deviation of
    s_ij = scale 2^-11 / sqrt(3) (sum_d q_d^2 k_d^2)^(1/2), independently from query to query, and the weights' error has the
    norm (sum_ij p_ij^2 s_ij^2)^(1/2); one and a half times that, and what split operands leave, is the bound. A single term
    is off by at most scale 2^-11 sum |q_d k_d| of itself."""
    L, hq, hkv, w0, wp = 2100, 8, 1, 300, 700
    g = si.generator(77)
    q, k = torch.randn(L, hq, 128, generator=g).bfloat16(), torch.randn(L, hkv, 128, generator=g).bfloat16()
    x, size = scores(q.double().numpy(), k.double().numpy(), w0, wp, si.FREQ_INTERP, False)
    m = x.max(2)
    l = (m + np.log(np.exp(x - m[..., None]).sum(2))).astype(np.float32)
    p = np.exp(x - l[..., None].astype(np.float64))
    want = p.sum((0, 1))
    # under any rotation |q_d k_d| sums, and its squares sum, to at most those of the pairs' lengths
    pair = [np.linalg.norm(np.stack([y[..., :64], y[..., 64:]]), axis=0).reshape(-1, 64) for y in (q.double().numpy(), k.double().numpy())]
    term = 2.0 ** -11 / math.sqrt(128) * (pair[0] @ pair[1].T).max()
    spread2 = 2.0 ** -22 / (3 * 128) * (pair[0] ** 2 @ (pair[1] ** 2).T).reshape(L, hq, L).transpose(1, 0, 2)
    cu = torch.tensor([0, L], dtype=torch.int32).cuda()
    got = bfl.bifocal_key_weights(q.cuda(), k.cuda(), torch.from_numpy(l).cuda(), cu, L, L, w0=w0, w_pretrained=wp, theta=THETA)
    assert bfl.last_device_error() == 0
    err = got[0].cpu().double().numpy() - want
    assert np.all(np.abs(err) <= (term + EPS * size + 4e-6) * want)
    bound = 1.5 * math.sqrt((p ** 2 * spread2).sum()) + (EPS * size / 16 + 1e-6) * np.linalg.norm(want)
    assert bound <= 2.7e-5 * np.linalg.norm(want)  # tight enough to see the keys' low parts missing (3e-5)
    assert np.linalg.norm(err) <= bound


def test_sum_is_the_number_of_queries():
    """With the prefill's own log-sum-exps the weights of a sequence sum to its queries times the group."""
    lens = [900, 350]
    g = si.generator(4)
    q, k, v = (torch.randn(1250, h, 128, generator=g).bfloat16().cuda() for h in (8, 2, 2))
    cu = torch.tensor([0, 900, 1250], dtype=torch.int32).cuda()
    kw = dict(w0=200, w_pretrained=300, theta=THETA)
    _, lse = bfl.bifocal_prefill_packed(q, k, v, cu, 900, **kw)
    got = bfl.bifocal_key_weights(q, k, lse, cu, 900, 500, **kw).double()
    for b, n in enumerate(lens):
        total = got[:, cu[b]:cu[b + 1]].sum(1)
        assert torch.all((total / (4 * min(n, 500)) - 1).abs() < 1e-3)  # the LSE's own bound


def test_bad_boundaries_and_pages_are_reported():
    g = si.generator(4)
    q, k = torch.randn(100, 4, 128, generator=g).bfloat16().cuda(), torch.randn(100, 2, 128, generator=g).bfloat16().cuda()
    lse = torch.full((4, 100), 4.0, device="cuda")
    kw = dict(w0=200, w_pretrained=300, theta=THETA)
    out = torch.full((2, 100), -3.0, device="cuda")
    for cu in ([0, 60, 50], [0, 101], [-1, 60], [0, 90]):
        bfl.bifocal_key_weights(q, k, lse, torch.tensor(cu, dtype=torch.int32).cuda(), 80, 10, kweight=out, **kw)
        assert bfl.last_device_error() == bfl.STATUS_INDEX and torch.all(out == -3)
    cu = torch.tensor([0, 80], dtype=torch.int32).cuda()
    want = bfl.bifocal_key_weights(q, k, lse, cu, 80, 10, **kw)[:, :80]
    table = torch.tensor([[1, 77, 0]], dtype=torch.int32).cuda()
    out = torch.full((2, 96), -3.0, device="cuda")
    bfl.bifocal_key_weights(q, k, lse, cu, 80, 10, kweight=out, page_size=32, block_table=table, **kw)
    assert bfl.last_device_error() == bfl.STATUS_INDEX
    assert torch.equal(out[:, 32:64], want[:, :32]) and torch.equal(out[:, :16], want[:, 64:]) and torch.all(out[:, 64:] == -3)


LONG = [
    # lens (of several, some have more than 16384 (query, head) rows and some fewer), hq, hkv, D, dtype, w0, w_pretrained, mode, q's size
    ([2100, 300], 8, 1, 128, torch.bfloat16, 300, 700, si.FREQ_INTERP, 1),
    ([2100], 8, 1, 128, torch.bfloat16, 300, 700, si.FREQ_INTERP, 4),
    ([150, 2070], 8, 1, 128, torch.float32, 0, 500, si.POS_ALIAS, 3),
    ([2100, 1], 8, 1, 64, torch.bfloat16, 1000, 300, si.POS_ALIAS, 3),
    ([2064], 16, 2, 64, torch.float32, 513, 1000, si.FREQ_INTERP, 1),
    ([700, 129], 6, 2, 128, torch.float32, 200, 300, si.FREQ_INTERP, 1),
]


@pytest.mark.parametrize("case", range(len(LONG)))
def test_every_key_over_all_queries(case):
    """Every single weight over all queries of long prompts is as exact as over few: the last keys too, which few
    queries see, and under peaked scores (q of three and four times the size). To the tolerance above comes the rounding of
    -lse log2(e), 2^-23 of it, which larger scores make larger than 1e-6."""
    lens, hq, hkv, D, dtype, w0, wp, mode, big = LONG[case]
    g = si.generator(700 + case)
    T = sum(lens)
    q, k = ((big if h == hq else 1) * torch.randn(T, h, D, generator=g) for h in (hq, hkv))
    q, k = q.to(dtype), k.to(dtype)
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    lse, want, tol = torch.empty(hq, T), [], []
    for b, n in enumerate(lens):
        s = slice(cu[b], cu[b] + n)
        x, size = scores(q[s].double().numpy(), k[s].double().numpy(), w0, wp, mode, False)
        m = x.max(2)
        l = (m + np.log(np.exp(x - m[..., None]).sum(2))).astype(np.float32)
        lse[:, s] = torch.from_numpy(l)
        x -= l[..., None].astype(np.float64)
        want.append(np.exp(x, out=x).sum(1).reshape(hkv, hq // hkv, n).sum(1))
        tol.append(EPS * size + 4e-6 + 2.0 ** -23 * np.abs(l).max())
    got = bfl.bifocal_key_weights(q.cuda(), k.cuda(), lse.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), max(lens),
                                  max(lens), w0=w0, w_pretrained=wp, theta=THETA, mode=mode)
    assert bfl.last_device_error() == 0
    got = got.cpu().double().numpy()
    for b, n in enumerate(lens):
        rel = np.abs(got[:, cu[b]:cu[b] + n] - want[b]) / np.maximum(want[b], 1e-30)
        worst = int(rel.max(0).argmax())
        assert np.all(rel * want[b] <= tol[b] * want[b] + 1e-30), (b, n, worst, rel.max(), tol[b])
