"""bifocal_cache_evict against a slot-by-slot reference: the pools, positions, weights and lengths after the
call are equal to the reference's bit for bit, everywhere (rows that must not change included)."""
import numpy as np
import pytest
import torch

import rope_context_extension_bifocal_b200 as bfl
import seeded_inputs as si
from tests.kept_ref import choose, moves, page_table, row_of

pytestmark = pytest.mark.gpu


def make(lens, hkv, D, page, seed, kind, positions="random"):
    g = si.generator(seed)
    table, pages = page_table(lens, page, g)
    rows = pages * page
    s = {"table": table, "rows": rows, "kc": torch.randn(rows, hkv, D, generator=g).bfloat16(),
         "vc": torch.randn(rows, hkv, D, generator=g).bfloat16(),
         "kpos": torch.full((hkv, rows), -7, dtype=torch.int32), "kw": torch.full((hkv, rows), float("nan"))}
    newest = []
    for b, n in enumerate(lens):
        span = 2 * n + 3
        newest.append(span)
        for h in range(hkv):
            pos = torch.randperm(span + 1, generator=g)[:n].int()
            if positions == "sorted":
                pos = pos.sort()[0]
            if kind == "lognormal":
                w = torch.exp(2 * torch.randn(n, generator=g))
            elif kind == "ties":
                w = torch.randint(0, 3, (n,), generator=g).float()
            elif kind == "equal":
                w = torch.zeros(n)
            else:  # every special value
                w = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 1e-45, 3e38, -1.0, 1.0, 1.0000001])
                w = w[torch.randint(0, len(w), (n,), generator=g)]
            for t in range(n):
                r = row_of(table, page, b, t)
                s["kpos"][h, r], s["kw"][h, r] = pos[t], w[t]
    s["newest"] = torch.tensor(newest, dtype=torch.int32)
    return s


def reference(s, lens, hkv, page, budget, recent, sink, dst=None):
    kc, vc, kpos, kw = (s[x].clone() for x in ("kc", "vc", "kpos", "kw"))
    for b, n in enumerate(lens):
        src = [row_of(s["table"], page, b, t) for t in range(n)]
        for h in range(hkv):
            kept = choose(s["kpos"][h, src].tolist(), s["kw"][h, src].tolist(), int(s["newest"][b]), min(n, budget), recent, sink)
            for f, t in moves(kept, n, dst is None):
                to = row_of(s["table"] if dst is None else dst, page, b, t)
                kc[to, h], vc[to, h], kpos[h, to], kw[h, to] = (s["kc"][src[f], h], s["vc"][src[f], h], s["kpos"][h, src[f]],
                                                                s["kw"][h, src[f]])
    return kc, vc, kpos, kw


def same(a, b):
    return torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32), b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))


def run(s, lens, page, budget, recent, sink, max_len=None, dst=None, alias=False):
    dev = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in s.items()}
    seq = torch.tensor(lens, dtype=torch.int32).cuda()
    new = bfl.bifocal_cache_evict(dev["kc"], dev["vc"], dev["kpos"], dev["kw"], page, dev["table"], seq, dev["newest"],
                                  max_len or max(max(lens), 1), budget, recent=recent, sink=sink,
                                  dst_block_table=None if dst is None else dst.cuda(), new_lens=seq if alias else None)
    return [dev[x].cpu() for x in ("kc", "vc", "kpos", "kw")], new.cpu()


CASES = [
    # lens, hkv, D, page, budget, recent, sink, weights, positions
    ([1], 1, 128, 16, 1, 0, 0, "lognormal", "sorted"),
    ([5, 0, 1, 9], 2, 64, 4, 3, 1, 1, "ties", "random"),
    ([100, 33, 64, 300], 3, 128, 16, 64, 10, 4, "special", "random"),
    ([700, 650], 2, 64, 1, 100, 0, 0, "equal", "random"),
    ([700, 650], 2, 128, 48, 649, 649, 0, "lognormal", "sorted"),
    ([1500, 31, 1025], 1, 128, 16, 700, 64, 8, "ties", "sorted"),
    ([5000, 4097], 2, 64, 64, 2000, 100, 4, "ties", "sorted"),       # two CTAs a segment
    ([9000, 12000], 1, 64, 16, 5000, 0, 100, "special", "random"),   # four
    ([17001, 20, 16385], 1, 64, 64, 1000, 16, 2, "lognormal", "sorted"),  # eight
]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_reference(case, in_place):
    lens, hkv, D, page, budget, recent, sink, kind, positions = CASES[case]
    s = make(lens, hkv, D, page, 40 + case, kind, positions)
    dst = None
    if not in_place:
        dst, more = page_table([min(n, budget) for n in lens], page, si.generator(case))
        dst = torch.where(dst >= 0, dst + s["rows"] // page, dst)
        grow = more * page
        for x in ("kc", "vc"):
            s[x] = torch.cat([s[x], torch.full((grow, hkv, D), 5.0, dtype=torch.bfloat16)])
        s["kpos"] = torch.cat([s["kpos"], torch.full((hkv, grow), -9, dtype=torch.int32)], 1)
        s["kw"] = torch.cat([s["kw"], torch.full((hkv, grow), 2.5)], 1)
        s["rows"] += grow
    want = reference(s, lens, hkv, page, budget, recent, sink, dst)
    got, new = run(s, lens, page, budget, recent, sink, dst=dst, alias=in_place)
    assert bfl.last_device_error() == 0
    assert new.tolist() == [min(n, budget) for n in lens]
    for a, b, name in zip(got, want, ("kcache", "vcache", "kpos", "kweight")):
        assert same(a, b), name


def test_more_slots_than_shared_memory_holds():
    """Over 8 * 40960 slots the keys are read again in every pass instead of being kept."""
    n, budget = 8 * 40960 + 777, 50000
    g = si.generator(1)
    w = torch.randint(0, 5000, (n,), generator=g).float()
    kpos = torch.arange(n, dtype=torch.int32)
    kc = torch.arange(n, dtype=torch.int32).view(torch.bfloat16).view(n, 1, 2).repeat(1, 1, 32).cuda()
    vc, dk, dw = kc.clone(), kpos.view(1, n).cuda(), w.view(1, n).cuda()
    seq, newest = torch.tensor([n], dtype=torch.int32).cuda(), torch.tensor([n - 1], dtype=torch.int32).cuda()
    table = torch.zeros(1, 1, dtype=torch.int32).cuda()
    bfl.bifocal_cache_evict(kc, vc, dk, dw, n, table, seq, newest, n, budget, recent=100, sink=4, new_lens=seq)
    assert bfl.last_device_error() == 0 and int(seq) == budget
    key = w.double().clone()
    key[:4] = key[-100:] = np.inf
    order = torch.argsort(key, dim=0, descending=True, stable=True)[:budget].sort()[0]
    want = torch.arange(n)
    holes = torch.ones(budget, dtype=torch.bool)
    holes[order[order < budget]] = False
    want[:budget][holes] = order[order >= budget]
    assert torch.equal(dk[0].cpu().long(), want)
    assert torch.equal(kc[:, 0, :2].cpu().contiguous().view(torch.int32).view(-1).long(), want)
    assert torch.equal(dw[0].cpu(), w[want])


def test_in_place_twice_changes_nothing():
    lens = [300, 40]
    s = make(lens, 2, 128, 16, 3, "lognormal", "sorted")
    got, new = run(s, lens, 16, 100, 10, 2)
    t = {**s, **dict(zip(("kc", "vc", "kpos", "kw"), got))}
    again, new2 = run(t, new.tolist(), 16, 100, 10, 2)
    assert new2.tolist() == new.tolist() and all(same(a, b) for a, b in zip(got, again))


def test_bad_lengths_and_pages_are_reported():
    lens = [40, 60, 50]
    s = make(lens, 2, 128, 16, 4, "lognormal")
    want = reference(s, [0, 60, 0], 2, 16, 20, 4, 0)
    got, new = run(s, [61, 60, -2], 16, 20, 4, 0, max_len=60)
    assert bfl.last_device_error() == bfl.STATUS_INDEX
    assert new.tolist() == [61, 20, -2]
    assert all(same(a, b) for a, b in zip(got, want))
    # a page outside the pool: its slots rank last, are not moved, and nothing outside the pool is touched
    s["table"][1, 1] = 1 << 20
    got, new = run(s, lens, 16, 20, 4, 0)
    assert bfl.last_device_error() == bfl.STATUS_INDEX and new.tolist() == [20, 20, 20]
    for b in (0, 2):
        for x, y in zip(got, reference(s, [n if i == b else 0 for i, n in enumerate(lens)], 2, 16, 20, 4, 0)):
            r = [row_of(s["table"], 16, b, t) for t in range(lens[b])]
            assert same((x[r] if x.dtype == torch.bfloat16 else x[:, r]).contiguous(),
                        (y[r] if y.dtype == torch.bfloat16 else y[:, r]).contiguous())


def test_captured_and_replayed():
    lens = [900, 1300]
    s = make(lens, 2, 128, 16, 6, "lognormal", "sorted")
    want = reference(s, lens, 2, 16, 256, 16, 4)
    dev = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in s.items()}
    seq = torch.tensor(lens, dtype=torch.int32).cuda()
    ws = torch.empty(bfl.cache_evict_workspace_size(2, 2, 1300, 256), dtype=torch.uint8, device="cuda")

    def call():
        bfl.bifocal_cache_evict(dev["kc"], dev["vc"], dev["kpos"], dev["kw"], 16, dev["table"], seq, dev["newest"], 1300, 256,
                                recent=16, sink=4, new_lens=seq, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):  # the second replay starts from the original contents again
        for x in ("kc", "vc", "kpos", "kw"):
            dev[x].copy_(s[x])
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert seq.tolist() == [256, 256]
        assert all(same(dev[x].cpu(), w) for x, w in zip(("kc", "vc", "kpos", "kw"), want))


CLUSTERS = [
    # lens, max_len (a CTA for every 16384 slots of it, up to eight), page, budget, recent, sink, weights
    ([20000, 300, 16384], 20000, 64, 3000, 100, 4, "ties"),         # two CTAs a segment
    ([33000, 1, 0, 32], 33000, 16, 9000, 0, 2, "special"),          # four
    ([50001, 17000], 50001, 48, 17000, 1000, 0, "ties"),
    ([66000, 40000], 66000, 128, 20000, 64, 16, "equal"),           # eight
    ([140000], 140000, 64, 70001, 500, 4, "ties"),
    ([70007], 100000, 64, 33, 16, 1, "special"),
    ([5, 700, 4097, 90], 140000, 64, 300, 20, 4, "ties"),           # a bound far above the lengths: most CTAs have no slot
]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("case", range(len(CLUSTERS)))
def test_segments_of_several_ctas_with_their_keys_resident(case, in_place):
    """Two, four and eight CTAs a segment, each with its keys in shared memory, with ties and special values across their
    borders: bit for bit a stable sort's choice."""
    lens, max_len, page, budget, recent, sink, kind = CLUSTERS[case]
    hkv, D = 2, 64
    g = si.generator(80 + case)
    table, pages = page_table(lens, page, g)
    width = -(-max_len // page)
    table = torch.cat([table, torch.full((len(lens), max(0, width - table.shape[1])), -1, dtype=torch.int32)], 1)
    to_table, rows = table, pages * page
    if not in_place:
        to_table, more = page_table([min(n, budget) for n in lens], page, g)
        to_table = torch.cat([to_table, torch.full((len(lens), -(-budget // page) - to_table.shape[1]), -1, dtype=torch.int32)], 1)
        to_table = torch.where(to_table >= 0, to_table + pages, to_table)
        rows += more * page
    words = torch.arange(rows * hkv, dtype=torch.int32).view(rows, hkv, 1)  # each row its own contents
    kc = words.repeat(1, 1, D // 2).view(torch.bfloat16).clone()
    vc = (~words).repeat(1, 1, D // 2).view(torch.bfloat16).clone()
    kpos, kw = torch.full((hkv, rows), -7, dtype=torch.int32), torch.full((hkv, rows), float("nan"))
    special = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 1e-45, 3e38, -1.0, 1.0, 1.0000001])
    newest = torch.tensor([2 * n + 3 for n in lens], dtype=torch.int32)

    def at(t, b, n):
        slot = torch.arange(n)
        return t[b, slot // page].long() * page + slot % page

    want = None
    for b, n in enumerate(lens):
        for h in range(hkv):
            kpos[h, at(table, b, n)] = torch.randperm(2 * n + 4, generator=g)[:n].int()
            kw[h, at(table, b, n)] = {"ties": lambda: torch.randint(0, 3, (n,), generator=g).float(), "equal": lambda: torch.zeros(n),
                                      "special": lambda: special[torch.randint(0, len(special), (n,), generator=g)]}[kind]()
    want = [t.clone() for t in (kc, vc, kpos, kw)]
    for b, n in enumerate(lens):
        m, src, dst = min(n, budget), at(table, b, n), at(to_table, b, min(n, budget))
        for h in range(hkv):
            pos, w = kpos[h, src], kw[h, src]
            key = w.double().nan_to_num(nan=-np.inf, posinf=1e300, neginf=-np.inf)
            key[(pos < sink) | (pos > int(newest[b]) - recent)] = np.inf
            kept = torch.argsort(key, descending=True, stable=True)[:m].sort()[0]
            if in_place:
                hole = torch.ones(m, dtype=torch.bool)
                hole[kept[kept < m]] = False
                f, t = src[kept[kept >= m]], src[:m][hole]
            else:
                f, t = src[kept], dst
            for new, old in zip(want[:2], (kc, vc)):
                new[t, h] = old[f, h]
            for new, old in zip(want[2:], (kpos, kw)):
                new[h, t] = old[h, f]
    dev = [t.cuda() for t in (kc, vc, kpos, kw)]
    seq = torch.tensor(lens, dtype=torch.int32).cuda()
    new = bfl.bifocal_cache_evict(*dev, page, table.cuda(), seq, newest.cuda(), max_len, budget, recent=recent, sink=sink,
                                  dst_block_table=None if in_place else to_table.cuda())
    assert bfl.last_device_error() == 0 and new.tolist() == [min(n, budget) for n in lens]
    for got, ref, name in zip(dev, want, ("kcache", "vcache", "kpos", "kweight")):
        assert same(got.cpu(), ref), name
