"""token_logprobs on a B200 against log_softmax in 64 bits.

Bounds: the others' sum s = sum e^(x-m) is a chain of at most V/128 + 64 additions per
thread and join, each within 2^-24 of a partial sum of positive terms, on terms that
carry 2^-21 of exp and of x - m scaled: relative at most 2^-21 + (V/128 + 64) 2^-24
< 2^-13 for V <= 2^18.  log1p passes that on at most as it is, so
|logprob - ref| <= 2^-13 s/(1+s) + 2^-22 |ref|; entropy = log1p(s) - t/(1+s) with the same
relative error in both terms: <= 2^-12 H + 2^-13 s/(1+s) covers it.  Ranks and ids are exact.
"""
import math

import pytest
import torch

from persistent_decode_b200 import XlpkError, _abi, token_logprobs

pytestmark = pytest.mark.gpu


def order(x):
    """Indices of a row in descending order: NaN first, ties by the lower index."""
    key = x.float().clone()
    nan = key.isnan()
    key[nan] = 0
    idx = torch.arange(x.numel())
    by = sorted(idx.tolist(), key=lambda i: (0 if nan[i] else 1, -float(key[i]), i))
    return by


def check(x, tok, r, k):
    """x [R][V] on the host."""
    R, V = x.shape
    xd = x.double()
    for i in range(R):
        t = int(tok[i])
        by = order(x[i])
        if k:
            assert r.top_ids[i].tolist() == by[:k]
        assert int(r.rank[i]) == (by.index(t) if 0 <= t < V else -1)
        if bool(x[i].isnan().any()) or bool((x[i] == math.inf).any()):
            assert math.isnan(r.logprob[i]) and math.isnan(r.entropy[i])
            if k:
                assert bool(r.top_logprobs[i].isnan().all())
            continue
        m = xd[i].max()
        if m == -math.inf:
            assert float(r.entropy[i]) == 0 and (not k or bool((r.top_logprobs[i] == -math.inf).all()))
            assert float(r.logprob[i]) == -math.inf if 0 <= t < V else math.isnan(r.logprob[i])
            continue
        e = torch.exp(xd[i] - m)
        e[by[0]] = 0
        s = e.sum()          # of all but the first maximum: 1 + s would round it away
        e[by[0]] = 1
        lp = xd[i] - m - torch.log1p(s)
        H = -(torch.where(e > 0, e * lp, 0.0)).sum() / (1 + s)
        slack = 2.0 ** -13 * float(s / (1 + s)) + 1e-30
        if 0 <= t < V:
            got, want = float(r.logprob[i]), float(lp[t])
            assert got == want or abs(got - want) <= slack + 2.0 ** -22 * abs(want), (got, want)
        else:
            assert math.isnan(r.logprob[i])
        assert abs(float(r.entropy[i]) - float(H)) <= slack + 2.0 ** -12 * float(H)
        if k:
            want = lp[by[:k]].tolist()
            for a, b in zip(r.top_logprobs[i].tolist(), want):
                assert a == b or abs(a - b) <= slack + 2.0 ** -22 * abs(b)


def run(x, tok, k, **kw):
    r = token_logprobs(x.cuda(), torch.tensor(tok, dtype=torch.int32, device="cuda"), top_k=k, **kw)
    return type(r)(*(f.cpu() if f is not None else None for f in r))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("R,V,k", [(1, 1, 1), (3, 2, 2), (4, 31, 31), (2, 64, 64), (5, 100, 0), (3, 1023, 64), (2, 4096, 20),
                                   (1, 32000, 5), (7, 8193, 1), (2, 128256, 64), (400, 257, 3), (3, 200003, 17)])
def test_matches_the_definition(cuda_device, R, V, k, dtype):
    g = torch.Generator().manual_seed(V + R)
    x = (torch.randn(R, V, generator=g) * 3).to(dtype)
    tok = [(i * 7919 + V - 1) % V for i in range(R)]
    check(x, tok, run(x, tok, k), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("V", [70, 5000, 40000])
def test_masks_ties_and_infinities(cuda_device, V, dtype):
    g = torch.Generator().manual_seed(V)
    low = torch.finfo(dtype).min
    base = (torch.randn(V, generator=g) * 2).to(dtype)
    rows = []

    def row(f):
        x = base.clone()
        f(x)
        rows.append(x)

    row(lambda x: x.fill_(-math.inf))                            # nothing is left
    row(lambda x: x.fill_(low))                                  # uniform over the lowest value
    row(lambda x: x.fill_(1.5))                                  # all the same: ids in order
    row(lambda x: x[:-1].fill_(-math.inf))                       # one token is left, the last
    row(lambda x: x[1:].fill_(low))
    row(lambda x: x[::3].fill_(-math.inf))
    row(lambda x: x[V // 2:].fill_(low))
    row(lambda x: x.copy_((torch.arange(V) % 5).to(dtype)))      # long ties across every part of the row
    row(lambda x: x.copy_(torch.arange(V, dtype=torch.float32).to(dtype)))          # ascending
    row(lambda x: x.copy_(-torch.arange(V, dtype=torch.float32).to(dtype)))         # descending
    row(lambda x: x[7].fill_(math.inf))
    row(lambda x: x[11].fill_(math.nan))
    row(lambda x: (x[::2].fill_(math.nan), x[1].fill_(math.inf)))
    row(lambda x: x.copy_(torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0).to(dtype)))   # -0 ties with +0
    row(lambda x: x[V - 2].fill_(40.0))                          # a nearly certain token
    x = torch.stack(rows)
    for tok in ([0] * len(rows), [V - 1] * len(rows), [V - 2, 11, 7] * (len(rows) // 3), [-1, V, 5] * (len(rows) // 3)):
        for k in (0, 64):
            check(x, tok, run(x, tok, k), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_large_logits_of_one_thread(cuda_device, dtype):
    # every large logit falls to the vectors that one thread of a part reads, so that what the other
    # threads have bounds the alternatives far below them, and more pass that bound than are ranked
    V, g = 700001, torch.Generator().manual_seed(11)
    x = torch.randn(2, V, generator=g)
    n = 16 // dtype.itemsize
    vec = torch.arange(V) // n
    x[:, vec % 256 == 5] += 60
    x = x.to(dtype)
    for k in (5, 64):
        check(x, [7, V - 1], run(x, [7, V - 1], k), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_nan_nearly_everywhere(cuda_device, dtype):
    x = torch.full((2, 9001), math.nan, dtype=dtype)
    x[:, 100:103] = torch.tensor([1.0, 2.0, 3.0]).to(dtype)
    check(x, [101, 8999], run(x, [101, 8999], 64), 64)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("low", [-1e4, -1e9, -3e9, -1e10, -1e12, -1e15, -1e30, -2e30, -1e35, -1e38])
def test_masks_of_finite_values(cuda_device, low, dtype):
    # masks that are neither -inf nor the type's lowest value; they are so far below the others, and
    # so far from each other, that their weights are exactly 0 in 64 bits too
    V, g = 40000, torch.Generator().manual_seed(12)
    base = (torch.randn(V, generator=g) * 2).to(dtype)
    rows = []

    def row(f):
        x = base.clone()
        f(x)
        rows.append(x)

    row(lambda x: x.fill_(low))                                  # nothing else is left: uniform
    row(lambda x: x[:-1].fill_(low))                             # the last token alone
    row(lambda x: x[1:].fill_(low))
    row(lambda x: x[:V // 2].fill_(low))                         # whole rounds of every thread, then the others
    row(lambda x: x[V // 2:].fill_(low))
    row(lambda x: x[::2].fill_(low))
    row(lambda x: x.copy_(torch.where(torch.rand(V, generator=g) < 0.999, low, base.float()).to(dtype)))
    row(lambda x: x.copy_((low * (1 + torch.arange(V) % 3)).to(dtype)))     # masked more than once: uniform over every third
    row(lambda x: x[7].fill_(-low))                              # as far out on the other side
    row(lambda x: x.copy_((-low * (1 + torch.arange(V) // 5000)).to(dtype)))
    x = torch.stack(rows)
    for tok in ([0] * len(rows), [V - 1] * len(rows), [7] * len(rows)):
        check(x, tok, run(x, tok, 0), 0)
    check(x, tok, run(x, tok, 64), 64)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("V,std", [(7, 1.0), (100, 0.1), (1023, 3.0), (4096, 0.5), (4096, 8.0)])
def test_digits_of_short_rows(cuda_device, V, std, dtype):
    """Bounds by the additions that rows this short take.  Of w = e^(x-m) = 2^y: the exponential 2^-22, the
    rounding of y and of log2(e) 2^-23 |y| together, of which the weighted mean is log2(V) at most; of a sum
    of V terms over 256 threads: V/256 + 16 in a thread, 5 and 16 across threads and warps, 2^-24 each; the
    factor that moves it to m: 2^-22.  So r = 2^-21 + 2^-23 log2(V) + (V/256 + 37) 2^-24 for the others' sum s.
    log1p passes on r s / (1+s) and adds its own 2^-23, x - m and the difference 2^-24 each of |logprob| or less:
    r s / (1+s) + 2^-22 |logprob|.  The mean of |x - m|, M, carries r twice (numerator, denominator) and 2^-23."""
    g = torch.Generator().manual_seed(V)
    R = 64
    x = (torch.randn(R, V, generator=g) * std).to(dtype)
    tok = torch.randint(0, V, (R,), generator=g)
    k = min(V, 64)
    got = run(x, tok.tolist(), k)
    xd = x.double()
    lp = torch.log_softmax(xd, 1)
    p = lp.exp()
    s = p.amax(1).reciprocal() - 1
    M = (p * (xd.amax(1, keepdim=True) - xd)).sum(1)
    r = 2.0 ** -21 + 2.0 ** -23 * math.log2(V) + (V / 256 + 37) * 2.0 ** -24
    slack = r * s / (1 + s)
    want = lp.gather(1, tok[:, None])[:, 0]
    assert bool(((got.logprob.double() - want).abs() <= slack + 2.0 ** -22 * want.abs()).all())
    want = lp.gather(1, got.top_ids.long())
    assert bool(((got.top_logprobs.double() - want).abs() <= slack[:, None] + 2.0 ** -22 * want.abs()).all())
    want = -(p * lp).sum(1)
    bound = slack + 2.0 ** -22 * torch.log1p(s) + (2 * r + 2.0 ** -23) * M + 2.0 ** -24 * want
    assert bool(((got.entropy.double() - want).abs() <= bound).all())


def test_a_certain_token_keeps_its_small_logprob(cuda_device):
    # log p of the best token is -s with s = 9 e^-20: far below the step of 1, kept to relative 2^-13
    x = torch.zeros(1, 10)
    x[0, 4] = 20
    r = run(x, [4], 1)
    want = -9 * math.exp(-20)
    assert abs(float(r.logprob[0]) - want) <= 2.0 ** -13 * abs(want)
    assert abs(float(r.top_logprobs[0, 0]) - want) <= 2.0 ** -13 * abs(want)
    assert abs(float(r.entropy[0]) - 21 * 9 * math.exp(-20)) <= 2.0 ** -12 * 21 * 9 * math.exp(-20)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 7])
def test_rows_at_any_stride_and_offset(cuda_device, offset, dtype):
    V, R, pad = 1201, 4, 7
    g = torch.Generator().manual_seed(offset)
    flat = (torch.randn(R * (V + pad) + 16, generator=g) * 2).to(dtype)
    flat[:] = torch.where(torch.arange(flat.numel()) % (V + pad) < 3, 50.0, flat.float()).to(dtype)   # loud neighbours
    x = flat[offset:offset + R * (V + pad)].view(R, V + pad)[:, 3:3 + V]
    d = flat.cuda()[offset:offset + R * (V + pad)].view(R, V + pad)[:, 3:3 + V]
    tok = [0, V - 1, 600, 1]
    r = token_logprobs(d, torch.tensor(tok, dtype=torch.int32, device="cuda"), top_k=9)
    check(x, tok, type(r)(*(f.cpu() for f in r)), 9)
    one = token_logprobs(d[2], torch.tensor(tok[2], dtype=torch.int32, device="cuda"), top_k=9)    # a single row: no leading shape
    assert one.logprob.shape == () and one.top_ids.shape == (9,) and torch.equal(one.logprob, r.logprob[2])


def test_shapes_of_a_decode(cuda_device):
    x = torch.randn(5, 3, 4096, generator=torch.Generator().manual_seed(1)).cuda()
    tok = torch.randint(0, 4096, (5, 3), dtype=torch.int32).cuda()
    r = token_logprobs(x, tok, top_k=4)
    assert r.logprob.shape == (5, 3) and r.top_ids.shape == (5, 3, 4)
    f = token_logprobs(x.view(15, 4096), tok.view(15), top_k=4)
    for a, b in zip(r, f):
        assert torch.equal(a.reshape(-1), b.reshape(-1))
    r = token_logprobs(x[:0], tok[:0], top_k=4)
    assert r.logprob.shape == (0, 3) and r.top_ids.shape == (0, 3, 4)
    r = token_logprobs(x[:1].expand(2, -1, -1)[:, 0], tok[:2, 0].contiguous())     # one row read twice
    assert r.top_ids is None and r.logprob.shape == (2,)


def test_same_bits_every_time_and_in_graphs(cuda_device):
    x = torch.randn(9, 50001, generator=torch.Generator().manual_seed(2)).cuda()
    y = x.flip(0).contiguous()
    tok = torch.arange(9, dtype=torch.int32).cuda()
    want = [token_logprobs(z, tok, 20) for z in (x, y)]
    for _ in range(3):
        for a, b in zip(token_logprobs(x, tok, 20), want[0]):
            assert torch.equal(a, b)
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for z in (x, y):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(token_logprobs(z, tok, 20))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))
    st = torch.cuda.Stream()
    got = token_logprobs(x, tok, 20, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))


def test_offsets_past_32_bits(cuda_device):
    flat = torch.empty((1 << 32) + 5000, dtype=torch.bfloat16, device=cuda_device)
    x = flat.as_strided((3, 4099), (1 << 31, 1))
    host = (torch.randn(3, 4099, generator=torch.Generator().manual_seed(3)) * 2).to(torch.bfloat16)
    x.copy_(host)
    r = token_logprobs(x, torch.tensor([0, 4098, 17], dtype=torch.int32, device=cuda_device), top_k=7)
    check(host, [0, 4098, 17], type(r)(*(f.cpu() for f in r)), 7)


def test_refusals(cuda_device):
    x = torch.zeros(4, 100, device=cuda_device)
    tok = torch.zeros(4, dtype=torch.int32, device=cuda_device)
    for bad in (lambda: token_logprobs(x.half(), tok), lambda: token_logprobs(x, tok.long()), lambda: token_logprobs(x, tok[:3]),
                lambda: token_logprobs(x.t(), torch.zeros(100, dtype=torch.int32, device=cuda_device)),
                lambda: token_logprobs(x, tok.cpu()), lambda: token_logprobs(x[:, :0], tok),
                lambda: token_logprobs(x.view(2, 2, 100).transpose(0, 1), tok.view(2, 2))):
        with pytest.raises(ValueError):
            bad()
    for k, st in ((-1, _abi.XLPK_ERR_INVALID_ARG), (65, _abi.XLPK_ERR_UNSUPPORTED), (101, _abi.XLPK_ERR_INVALID_ARG)):
        with pytest.raises(XlpkError) as e:
            token_logprobs(x, tok, top_k=k)
        assert e.value.status == st
