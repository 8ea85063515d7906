"""The packed and eviction operators as a server launches them: captured and replayed with other contents, on a side
stream, two calls in flight on two streams, and twice with the same result."""
import pytest
import torch

import rope_context_extension_bifocal_b200 as bfl
import seeded_inputs as si

pytestmark = pytest.mark.gpu
KW = dict(w0=50, w_pretrained=64, theta=1e6)


def prompts(seed, lens, D=128, hq=4, hkv=2):
    g = si.generator(seed)
    T = sum(lens)
    x = [torch.randn(T, h, D, generator=g).bfloat16().cuda() for h in (hq, hkv, hkv)]
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda()
    return x, cu


def both(x, cu, max_len, stream=None):
    out, lse = bfl.bifocal_prefill_packed(*x, cu, max_len, stream=stream, **KW)
    return out, lse, bfl.bifocal_key_weights(x[0], x[1], lse, cu, max_len, 40, stream=stream, **KW)


@pytest.mark.parametrize("D,hq,hkv", [(128, 4, 2), (128, 3, 1), (64, 4, 2)])
def test_captured_and_replayed_with_other_lengths(D, hq, hkv):
    a, cu_a = prompts(1, [200, 1, 99], D, hq, hkv)
    b, cu_b = prompts(2, [30, 170, 100], D, hq, hkv)
    want = [both(a, cu_a, 200), both(b, cu_b, 200)]
    torch.cuda.synchronize()
    x, cu = [t.clone() for t in a], cu_a.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(x, cu, 200)
    for inputs, bounds, ref in ((b, cu_b, want[1]), (a, cu_a, want[0]), (b, cu_b, want[1])):
        for t, s in zip(x, inputs):
            t.copy_(s)
        cu.copy_(bounds)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, ref))
    assert bfl.last_device_error() == 0


def test_two_streams_and_repeats():
    a, cu_a = prompts(3, [700, 33])
    b, cu_b = prompts(4, [64, 500, 7])
    want = [both(a, cu_a, 700), both(b, cu_b, 700)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        r1 = both(a, cu_a, 700, stream=s1)
        r2 = both(b, cu_b, 700, stream=s2)
        s1.synchronize()
        s2.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(r1, want[0]))
        assert all(torch.equal(g, w) for g, w in zip(r2, want[1]))
    assert bfl.last_device_error() == 0


def test_many_short_sequences():
    """More sequences than a list of levels, threads or tiles holds at once, most of them one token."""
    g = si.generator(9)
    lens = [int(n) for n in torch.randint(0, 4, (3000,), generator=g)]
    x, cu = prompts(5, lens, 64, 2, 1)
    out, lse, w = both(x, cu, 3)
    assert bfl.last_device_error() == 0
    first = cu[:-1][torch.tensor(lens).cuda() > 0].long()
    assert torch.equal(out[first], x[2][first].expand(-1, 2, -1))  # a first token sees itself alone
    total = torch.zeros(3000, device="cuda").index_add_(0, torch.repeat_interleave(torch.arange(3000).cuda(), torch.tensor(lens).cuda()), w[0])
    assert torch.all((total - 2 * torch.tensor(lens).cuda()).abs() <= 2e-3 * torch.tensor(lens).cuda() + 1e-6)


def test_long_rows_of_one_sequence_in_a_large_batch():
    """A long sequence between short ones: its tiles spread over many levels of work."""
    lens = [1] * 40 + [2600] + [3] * 20
    x, cu = prompts(6, lens)
    out, lse, w = both(x, cu, 2600)
    s = slice(40, 2640)
    alone = both([t[s].contiguous() for t in x], torch.tensor([0, 2600], dtype=torch.int32).cuda(), 2600)
    assert torch.equal(out[s], alone[0]) and torch.equal(lse[:, s], alone[1]) and torch.equal(w[:, s], alone[2])
    assert bfl.last_device_error() == 0
