"""decode_attention on a B200 against the definition in 64 bits.

Bounds, per output element, with S = scale * sum_i |q_i k_i| (the largest over the
visible positions), A = sum_t p_t |v_t| and T visible positions:
 * a score is a sum of 3 x 8 products of MMAs at most (fp32 q in three bf16 terms, 128
   dims), each accumulated to 2^-22 of the partial sum, plus 2^-24 for the terms' remainder:
   |ds| <= 25 * 2^-22 S < 2^-17 S; as a factor on p that is e^ds, relative to the softmax's
   denominator twice that: 2^-16 S;
 * p carries 2^-21 of exp2 and of its scaling and 2^-16 of its split (two terms); sums over T
   positions lose 2^-22 each of T/16 times and once per warp or CTA joined: T 2^-26 + 2^-15 in all;
 * the result is rounded once: half a step of its type.
So |out - ref| <= A (2^-16 S + T 2^-26 + 2^-15) + eps/2 |ref|, and the same without A for lse (plus
its own fp32 rounding, 2^-24 |lse|).
"""
import math

import pytest
import torch

from persistent_decode_b200 import XlpkError, _abi, decode_attention

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def make(B, lens, H, KH, D, page, kv="bf16", io=torch.bfloat16, seed=0, capacity=None, std=1.0, hnd=True):
    """Inputs whose cache entries that no position names are NaN, as the caller's memory may be."""
    g = torch.Generator().manual_seed(seed)
    scale = 2.0 ** -5 if kv == "e4m3" else 1.0
    cap = capacity or max(max(lens), 1)
    P = page or cap
    cols = -(-cap // P)
    if page:
        used = [-(-n // P) for n in lens]
        n_pages = sum(used) + 2
        ids = torch.randperm(n_pages, generator=g).to(torch.int32)
        table, at = torch.full((B, cols), -1, dtype=torch.int32), 0
        table[:, 1::2] = 1 << 30                       # behind the sequence: anything
        for b in range(B):
            table[b, :used[b]] = ids[at:at + used[b]]
            at += used[b]
    else:
        n_pages, table = B, None

    def cache():
        vals = torch.randn(n_pages, KH, P, D, generator=g) * std
        seen = torch.zeros(n_pages, P, dtype=torch.bool)
        for b, n in enumerate(lens):
            t = torch.arange(n)
            seen[table[b, t // P].long() if page else torch.full_like(t, b), t % P] = True
        seen = seen[:, None, :, None]
        if kv == "e4m3":
            codes = (vals / scale).clamp(-448, 448).to(E4M3).view(torch.uint8)
            out = torch.where(seen, codes, 0x7f)
        else:
            out = torch.where(seen, vals.to(torch.bfloat16), float("nan"))
        if not hnd:     # positions outside heads in memory
            out = out.transpose(1, 2).contiguous().transpose(1, 2)
        return out.cuda()

    k, v = cache(), cache()
    if not hnd:
        assert k.stride(1) == D
    q = (torch.randn(B, H, D, generator=g) * std).to(io).cuda()
    return dict(q=q, k=k, v=v, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                table=None if table is None else table.cuda(), scale_kv=scale, P=P)


def values(x, scale):
    return (x.view(E4M3) if x.dtype == torch.uint8 else x).float().double() * scale


def reference(s, scale=None, window=0, sinks=0):
    """(out, lse, S, A) in 64 bits on the host."""
    q, lens = s["q"].double().cpu(), s["lens"].tolist()
    B, H, D = q.shape
    KH, P = s["k"].shape[1], s["P"]
    scale = 1 / math.sqrt(D) if scale is None else scale
    out, lse = torch.zeros(B, H, D, dtype=torch.float64), torch.full((B, H), -math.inf, dtype=torch.float64)
    S, A = torch.zeros(B, H, dtype=torch.float64), torch.zeros(B, H, D, dtype=torch.float64)
    k, v = values(s["k"], s["scale_kv"]).cpu(), values(s["v"], s["scale_kv"]).cpu()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        t = torch.arange(n)
        if window:
            t = t[(t >= n - window) | (t < sinks)]
        page = s["table"].cpu()[b, t // P].long() if s["table"] is not None else torch.full_like(t, b)
        for h in range(H):
            kk, vv = k[page, h * KH // H, t % P], v[page, h * KH // H, t % P]
            sc = (kk @ q[b, h]) * scale
            lse[b, h] = torch.logsumexp(sc, 0)
            p = torch.exp(sc - lse[b, h])
            out[b, h], A[b, h] = p @ vv, p @ vv.abs()
            S[b, h] = ((kk * q[b, h]).abs().sum(1) * scale).max()
    return out, lse, S, A


def check(s, got, lse, window=0, sinks=0, scale=None):
    ref, rlse, S, A = reference(s, scale, window, sinks)
    T = float(s["lens"].max()) if not window else window + sinks
    rel = 2.0 ** -16 * S + T * 2.0 ** -26 + 2.0 ** -15
    bound = A * rel[..., None] + torch.finfo(got.dtype).eps / 2 * ref.abs()
    err = (got.double().cpu() - ref).abs()
    assert bool((err <= bound + 1e-30).all()), float((err / (bound + 1e-30)).max())
    lse = lse.double().cpu()
    dead = rlse == -math.inf
    assert torch.equal(lse[dead], rlse[dead])
    assert bool(((lse - rlse).abs() <= rel + 2.0 ** -24 * rlse.abs())[~dead].all())


def call(s, **kw):
    return decode_attention(s["q"], s["k"], s["v"], s["lens"], s["table"], k_scale=s["scale_kv"], v_scale=s["scale_kv"],
                            return_lse=True, **kw)


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 129, 200, 777]


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,KH,D,page", [(4, 2, 64, 128), (32, 8, 128, 64), (28, 4, 128, 16), (16, 1, 128, 64),
                                         (3, 3, 64, 24), (10, 2, 64, 7), (12, 1, 64, 1), (22, 2, 128, 0), (8, 1, 128, 0),
                                         (9, 1, 128, 40)])
def test_matches_the_definition(cuda_device, H, KH, D, page, kv, io):
    s = make(len(LENS), LENS, H, KH, D, page, kv, io, seed=H + D + page)
    check(s, *call(s))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (100, 3), (64, 64), (50, 700), (2000, 4)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 0), (128, 24)])
def test_window_and_first_tokens(cuda_device, window, sinks, D, page, kv):
    s = make(len(LENS), LENS, 6, 2, D, page, kv, seed=window + sinks)
    if page:    # pages that no position sees are gone
        for b, n in enumerate(LENS):
            for j in range(-(-n // page)):
                if (j + 1) * page <= n - window and j * page >= sinks:
                    s["table"][b, j] = -1
                    # the reference skips them too: it looks up visible positions alone
    check(s, *call(s, window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("B,n", [(1, 40001), (2, 8193), (1, 1), (1, 16), (700, 3), (150, 130)])
def test_split_and_joined(cuda_device, B, n):
    # one long sequence spread over the whole GPU, and more sequences than it has SMs
    s = make(B, [n] * B, 4, 1, 64, 32, seed=n)
    check(s, *call(s))


@pytest.mark.parametrize("H,KH,D,kv,io", [(16, 1, 128, "bf16", torch.bfloat16), (16, 1, 128, "e4m3", torch.float32),
                                          (12, 1, 64, "bf16", torch.float32), (8, 2, 64, "e4m3", torch.bfloat16),
                                          (7, 1, 128, "bf16", torch.float32), (10, 2, 64, "e4m3", torch.float32)])
@pytest.mark.parametrize("B,most", [(300, 90), (170, 700), (2, 6000)])
def test_many_short_and_few_long_sequences(cuda_device, B, most, H, KH, D, kv, io):
    # segments that warps share, that CTAs share, and that are cut into pieces either way
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, most + 1, (B,), generator=g).tolist()
    lens[0] = most
    s = make(B, lens, H, KH, D, 48, kv, io, seed=B + H)
    check(s, *call(s))


def test_one_sequence_outlasts_all_others(cuda_device):
    s = make(400, [9000] + [3] * 399, 4, 2, 64, 16, seed=2)
    check(s, *call(s))


@pytest.mark.parametrize("H,KH,D,kv,io", [(16, 1, 128, "bf16", torch.float32), (16, 1, 128, "e4m3", torch.bfloat16),
                                          (9, 1, 64, "e4m3", torch.float32), (8, 1, 128, "bf16", torch.bfloat16)])
def test_short_segments_follow_each_other_in_one_cta(cuda_device, H, KH, D, kv, io):
    # one long sequence makes CTAs the workers; each of them then joins its warps' results for a dozen
    # segments of one tile, through the same scratch, one right after the other
    s = make(1500, [30000] + [1 + b % 16 for b in range(1499)], H, KH, D, 16, kv, io, seed=22)
    got, lse = call(s)
    check(s, got, lse)
    for _ in range(10):
        a, b = call(s)
        assert torch.equal(a, got) and torch.equal(b, lse)


def test_ragged_lengths_share_the_work(cuda_device):
    lens = [5, 9000, 0, 1, 333, 0, 2500, 16]
    s = make(len(lens), lens, 8, 2, 128, 64, "e4m3", torch.float32, seed=3)
    check(s, *call(s))


def test_peaked_scores_and_scale(cuda_device):
    # scores of hundreds, so that one position holds nearly all of the weight
    s = make(3, [40, 300, 1], 4, 2, 64, 16, std=6.0, seed=9)
    check(s, *call(s, scale=0.7), scale=0.7)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,H,KH,D", [(40, 8, 1, 64), (1500, 8, 1, 64), (300, 8, 2, 128), (40, 16, 1, 64), (300, 16, 1, 128),
                                      (200, 9, 1, 128), (300, 3, 3, 128)])
def test_positions_of_different_tiles_weigh_by_the_same_measure(cuda_device, B, H, KH, D, kv):
    """Two positions of five tiles carry all of the weight, the later one more of it; the ratio of their
    outputs is 2^(x0 - x1) whatever the softmax is measured from.  Scores are exact: one product with 1, of q
    whose 23 bits two fp16 terms hold, times a scale of which scale * log2(e) is 1 in fp32 (it is 2.8e-9
    off ln 2, which adds 8 x 2.8e-9).  So the ratio carries three exponentials (2^-22 each: both weights and
    the rescaling of the first), the split of both weights (two 11-bit terms: 2^-24 each), a rescaling and
    two products of the result (2^-24 each): 17 x 2^-24 and that, below 18 x 2^-24 (sums of the terms are exact).
    A term of q or p that is lost shows: the third of bf16 q leaves up to 2^-18 of 8, that of p 2^-18."""
    n = 80
    g = torch.Generator().manual_seed(31)
    x = -8 + torch.randint(1, 1 << 21, (B, H, 2), generator=g).double() * 2.0 ** -20
    x = x.sort(dim=2).values
    q = torch.zeros(B, H, D)
    q[..., :2], q[..., 2] = x.float(), -256.0
    assert torch.equal(q[..., :2].double(), x)
    k, v = torch.zeros(B, KH, n, D), torch.zeros(B, KH, n, D)
    k[:, :, :, 2] = 1
    for i, t in enumerate((5, n - 1)):
        k[:, :, t, 2], k[:, :, t, i], v[:, :, t, i] = 0, 1, 1
    k, v = ((t.to(E4M3).view(torch.uint8) if kv == "e4m3" else t.to(torch.bfloat16)).cuda() for t in (k, v))
    out = decode_attention(q.cuda(), k, v, torch.full((B,), n, dtype=torch.int32, device=cuda_device),
                           scale=float(torch.tensor(math.log(2)))).double().cpu()
    ratio = out[..., 0] / out[..., 1]
    want = torch.exp2(x[..., 0] - x[..., 1])
    assert float((ratio / want - 1).abs().max()) <= 18 * 2.0 ** -24


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("H,KH,D", [(8, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("power", [124, 101, 99, -99, -101, -117, -129])
def test_queries_of_any_size_over_e4m3(cuda_device, power, H, KH, D, io):
    # q near either end of fp32's range, with a scale that makes ordinary scores of it
    s = make(4, [1, 40, 333, 16], H, KH, D, 16, "e4m3", io, seed=power + 200)
    s["q"] = (s["q"].double() * 2.0 ** power).to(io)
    assert bool(s["q"].isfinite().all()) and float(s["q"].abs().max()) > 0
    scale = 2.0 ** (-power - 3)
    check(s, *call(s, scale=scale), scale=scale)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("H,KH,D", [(8, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("power", [12, 21, 23, 25, 27, 29, 31, 33, 50, 90])
def test_scores_of_any_finite_size(cuda_device, power, H, KH, D, io, kv):
    # The score of position t is 2^power x_t with whole x_t in -8 .. 8, but for one of 9: at these distances
    # (2^12 and more) it has all of the weight, whatever its sign and wherever it stands, and the output is
    # its v: to half a step of the output's type, and in fp32 what p's split (2^-24), the sums of its products
    # (2^-23 each of two), the sum of the terms, the quotient and the product (2^-24 each) add: 2^-21
    lens = [1, 40, 333, 700]
    s = make(len(lens), lens, H, KH, D, 0, kv, io, seed=power)
    g = torch.Generator().manual_seed(power)
    for sign in (1, -1):
        x = torch.randint(-8, 9, (len(lens), KH, s["P"]), generator=g)
        best = [int(torch.randint(0, n, (1,), generator=g)) for n in lens]
        if sign < 0:
            x = x.abs() - 30           # -30 .. -22
        for b, t in enumerate(best):
            x[b, :, t] = 9 if sign > 0 else -20
        k = torch.zeros(len(lens), KH, s["P"], D)
        k[..., 0], k[..., 1] = (x // 4).float(), (x % 4).float()       # x = 4 k0 + k1: exact in either type
        s["k"] = (k.to(E4M3).view(torch.uint8) if kv == "e4m3" else k.to(torch.bfloat16)).cuda()
        s["q"] = torch.zeros(len(lens), H, D, dtype=io, device=cuda_device)
        s["q"][..., 0], s["q"][..., 1] = 2.0 ** (power + 2), 2.0 ** power
        out, lse = decode_attention(s["q"], s["k"], s["v"], s["lens"], scale=1.0, v_scale=s["scale_kv"], return_lse=True)
        v = values(s["v"], s["scale_kv"]).cpu()
        want = torch.stack([v[b, :, t] for b, t in enumerate(best)]).repeat_interleave(H // KH, 1)
        slack = torch.finfo(io).eps / 2 + 2.0 ** -21
        assert bool(((out.double().cpu() - want).abs() <= slack * want.abs()).all())
        score = 2.0 ** power * (9 if sign > 0 else -20)
        # log2(e), its product with the score, ln 2, the product with that and the sum: five roundings; the
        # log of the weights' sum, of 1 or 2^10: two
        assert float((lse.double() - score).abs().max()) <= 5 * 2.0 ** -24 * abs(score) + 2 * 2.0 ** -24 * 10


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,D", [(4, 64), (4, 128), (16, 64), (12, 128)])
def test_long_sums_do_not_fall_behind(cuda_device, H, D, kv):
    """Sums of the tensor cores are cut off, not rounded: less than a step (2^-23) for each product added. Where
    all values are positive that is a bias, which grows with the positions that one warp sums up: here
    590 to 886 tiles of 16.
    Over at most 64 tiles (32, of up to 3 products each, with more than 8 heads) whose sum grows evenly from nothing
    it is below 64 (96) halves of a step, 2^-24, on average over the outputs; exponentials add 2^-22, the denominator's
    rounded sums and the rest 2^-22."""
    B, n = 1024, 16384
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn(1, 1, n, D, generator=g, device="cuda")
    v = 1 + torch.rand(1, 1, n, D, generator=g, device="cuda")
    k, v = (t.to(E4M3) if kv == "e4m3" else t.to(torch.bfloat16) for t in (k, v))
    q = torch.randn(B, H, D, generator=g, device="cuda")
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    out, _ = decode_attention(q, k.expand(B, -1, -1, -1), v.expand(B, -1, -1, -1), lens, return_lse=True)
    off = []
    for part, got in zip(q.split(64), out.split(64)):
        p = torch.softmax(torch.einsum("bhd,td->bht", part.double(), k[0, 0].double()) / math.sqrt(D), 2)
        off.append(got.double() / torch.einsum("bht,td->bhd", p, v[0, 0].double()) - 1)
    bias = float(torch.cat(off).mean())
    assert abs(bias) <= (64 if H <= 8 else 96) * 2.0 ** -24 + 2.0 ** -21, bias


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("trend", [20.0, -20.0, 0.0])
@pytest.mark.parametrize("B,H,KH,D,n", [(1024, 4, 1, 64, 16384), (400, 12, 1, 128, 16384), (2, 16, 8, 64, 262144), (2, 16, 8, 128, 200003),
                                       (2, 32, 2, 128, 400001)])
def test_long_sums_whose_maximum_moves(cuda_device, B, H, KH, D, n, trend, kv):
    # scores that rise or fall by 20 along the sequence, so that what a warp has added up is rescaled again and
    # again; warps as workers (many sequences), and CTAs (two)
    g = torch.Generator(device="cuda").manual_seed(7)
    k = torch.randn(1, 1, n, D, generator=g, device="cuda") * 0.5
    k[..., 0] = torch.linspace(0, trend / 2, n, device="cuda")
    v = torch.randn(1, 1, n, D, generator=g, device="cuda") + 1
    k, v = (t.to(E4M3) if kv == "e4m3" else t.to(torch.bfloat16) for t in (k, v))
    q = torch.randn(B, H, D, generator=g, device="cuda")
    q[..., 0] = 2
    lens = torch.randint(n // 2, n + 1, (B,), generator=g, device="cuda").int()
    lens[0] = n
    out, lse = decode_attention(q, k.expand(B, KH, -1, -1), v.expand(B, KH, -1, -1), lens, scale=1.0, return_lse=True)
    kk, vv = k[0, 0].double(), v[0, 0].double()
    for b in range(0, B, max(1, B // 16)):
        m = int(lens[b])
        sc = q[b].double() @ kk[:m].T
        S = (q[b].double().abs() @ kk[:m].abs().T).amax(1)
        want_lse = torch.logsumexp(sc, 1)
        p = torch.exp(sc - want_lse[:, None])
        want, Am = p @ vv[:m], p @ vv[:m].abs()
        # (a warp's or a CTA's sum of 64 tiles at a time, and these, each added to 2^-23: below T / 16 times that)
        rel = 2.0 ** -16 * S + m * 2.0 ** -26 + 2.0 ** -15
        assert bool(((out[b].double() - want).abs() <= Am * rel[:, None] + 2.0 ** -24 * want.abs()).all())
        assert bool(((lse[b].double() - want_lse).abs() <= rel + 2.0 ** -24 * want_lse.abs()).all())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,KH,D", [(8, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("size,scale", [(2.0 ** -100, 2.0 ** -100), (2.0 ** -120, 2.0 ** -149), (0.0, 2.0 ** 126), (1.0, 2.0 ** -149)])
def test_scores_that_vanish(cuda_device, size, scale, H, KH, D, kv):
    # scores of (next to) nothing, in rows whose last tile has hidden positions: every visible one weighs the same
    s = make(4, [1, 40, 333, 17], H, KH, D, 16, kv, torch.float32, seed=41)
    s["q"] = (s["q"].double() * size).float()
    check(s, *call(s, scale=scale, window=100, sinks=3), scale=scale, window=100, sinks=3)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("H,KH,D,page", [(8, 2, 64, 16), (8, 2, 128, 0), (5, 5, 128, 24), (16, 1, 64, 5)])
def test_stores_the_new_row(cuda_device, H, KH, D, page, io, kv):
    lens = [1, 16, 17, 0, 100, 24, 25]
    s = make(len(lens), lens, H, KH, D, page, kv, io, seed=21, capacity=128)
    g = torch.Generator().manual_seed(5)
    new = {n: (torch.randn(len(lens), KH, D, generator=g) * 20).to(io).cuda() for n in ("k", "v")}   # e4m3: some saturate
    want = {}
    for name in ("k", "v"):
        want[name] = s[name].clone()
        for b, n in enumerate(lens):
            if n:
                pg = int(s["table"][b, (n - 1) // s["P"]]) if page else b
                x = new[name][b].float() / s["scale_kv"]
                want[name][pg, :, (n - 1) % s["P"]] = x.clamp(-448, 448).to(E4M3).view(torch.uint8) if kv == "e4m3" \
                    else x.to(torch.bfloat16)
                s[name][pg, :, (n - 1) % s["P"]] = 0x7f if kv == "e4m3" else float("nan")   # whatever stood there
    got, lse = call(s, k_new=new["k"], v_new=new["v"])
    for name in ("k", "v"):      # that row, and nothing else
        assert torch.equal(s[name].view(torch.uint8), want[name].view(torch.uint8))
    check(s, got, lse)


def test_strided_operands(cuda_device):
    # q, k_new, v_new cut from one projection's output; out inside a wider buffer; cache [pages][positions][heads][d]
    lens, H, KH, D = [33, 70, 5], 8, 2, 64
    s = make(3, lens, H, KH, D, 16, seed=4, hnd=False)
    qkv = torch.randn(3, H + 2 * KH, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    s["q"], kn, vn = qkv[:, :H], qkv[:, H:H + KH], qkv[:, H + KH:]
    wide = torch.full((3, 2 * H, 2 * D), 7.0, dtype=torch.bfloat16, device=cuda_device)
    out = wide[:, ::2, :D]
    got, lse = call(s, k_new=kn, v_new=vn, out=out)
    assert got.data_ptr() == wide.data_ptr()
    check(s, got, lse)
    assert bool((wide[:, 1::2] == 7).all()) and bool((wide[:, ::2, D:] == 7).all())


def test_broadcast_query(cuda_device):
    s = make(4, [20, 30, 40, 50], 8, 2, 64, 16, seed=6)
    s["q"] = s["q"][:1].expand(4, -1, -1)
    check(s, *call(s))


def test_same_bits_every_time(cuda_device):
    s = make(5, [3000, 1, 700, 0, 64], 8, 2, 128, 64, seed=8)
    a, la = call(s)
    for _ in range(3):
        b, lb = call(s)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_bad_pages_and_lengths_are_reported(cuda_device):
    s = make(6, [200, 200, 200, 200, 200, 1], 8, 2, 64, 16, seed=12)
    ref, _ = call(s)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    call(s, status=status)
    assert int(status) == 0
    s["table"][1, 3] = s["k"].shape[0]
    s["table"][2, 12] = -1
    s["lens"][3] = 10 ** 9
    s["lens"][4] = -5
    got, lse = call(s, status=status)
    assert int(status) == _abi.XLPK_ERR_INVALID_ARG
    assert bool(got[1:5].isnan().all()) and bool(lse[1:5].isnan().all())
    assert torch.equal(got[[0, 5]], ref[[0, 5]])
    # a new row whose page is bad is stored nowhere
    k0 = s["k"].clone()
    new = torch.ones(6, 2, 64, dtype=torch.bfloat16, device=cuda_device)
    s["lens"][:] = torch.tensor([0, 0, 200, 10 ** 9, -5, 0], dtype=torch.int32)
    got, _ = call(s, k_new=new, v_new=new)
    assert torch.equal(s["k"].view(torch.uint8), k0.view(torch.uint8))
    assert bool(got[2:5].isnan().all()) and bool((got[[0, 1, 5]] == 0).all())


def test_captured_and_replayed_with_new_lengths(cuda_device):
    # two graphs of the same call, replayed side by side on two streams, with lengths changed in between
    s = make(4, [500, 300, 900, 1], 8, 2, 64, 32, seed=14)
    r = dict(s, q=s["q"].flip(0).contiguous())
    call(s)
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for x in (s, r):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(x))
        graphs.append(g)
    for lens in ([500, 300, 900, 1], [0, 299, 17, 1], [500, 16, 64, 1]):
        s["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        for _ in range(5):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for x, (o, l) in zip((s, r), outs):
            want, wl = call(x)
            assert torch.equal(o, want) and torch.equal(l, wl)


def test_on_another_stream(cuda_device):
    s = make(2, [700, 800], 4, 2, 64, 64, seed=15)
    want, _ = call(s)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, _ = call(s, stream=st)
    other, _ = call(s)
    st.synchronize()
    assert torch.equal(got, want) and torch.equal(other, want)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_offsets_past_32_bits(cuda_device, kv):
    # the same few pages at both ends of pools of more than 2^32 bytes
    small = make(2, [300, 77], 4, 1, 128, 64, kv, seed=17)
    want, _ = call(small)
    pages = (1 << 32) // (64 * 128 * small["k"].element_size()) + 1000
    n = small["k"].shape[0]
    where = torch.arange(n, device=cuda_device) + torch.where(torch.arange(n, device=cuda_device) % 2 == 0, pages - n, 0)
    big = dict(small)
    for name in ("k", "v"):
        big[name] = torch.empty((pages, *small[name].shape[1:]), dtype=small[name].dtype, device=cuda_device)
        big[name][where] = small[name]
    t = small["table"]
    big["table"] = torch.where((t >= 0) & (t < n), where[t.clamp(0, n - 1).long()].int(), t)
    got, _ = call(big)
    assert torch.equal(got, want)


def test_no_sequences(cuda_device):
    s = make(1, [5], 4, 2, 64, 16)
    got = decode_attention(s["q"][:0], s["k"], s["v"], s["lens"][:0], s["table"][:0])
    assert got.shape == (0, 4, 64)


@pytest.mark.parametrize("kv", [torch.bfloat16, torch.uint8], ids=["bf16", "e4m3"])
def test_a_pool_without_pages(cuda_device, kv):
    none = torch.empty((0, 2, 16, 64), dtype=kv, device=cuda_device)
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device=cuda_device)
    table = torch.zeros((3, 2), dtype=torch.int32, device=cuda_device)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    lens = torch.tensor([0, 20, 0], dtype=torch.int32, device=cuda_device)
    new = torch.ones(3, 2, 64, dtype=torch.bfloat16, device=cuda_device)
    for extra in ({}, dict(k_new=new, v_new=new)):
        status.zero_()
        out, lse = decode_attention(q, none, none, lens, table, status=status, return_lse=True, **extra)
        assert int(status) == _abi.XLPK_ERR_INVALID_ARG
        assert bool(out[1].isnan().all()) and bool((out[[0, 2]] == 0).all()) and bool((lse[[0, 2]] == -math.inf).all())


def test_refusals(cuda_device):
    s = make(2, [20, 30], 4, 2, 64, 16)
    q, k, v, lens, table = s["q"], s["k"], s["v"], s["lens"], s["table"]
    for bad in (lambda: decode_attention(q.half(), k, v, lens, table),
                lambda: decode_attention(q, k.half(), v.half(), lens, table),
                lambda: decode_attention(q, k, v[:1], lens, table),
                lambda: decode_attention(q, k, v, lens.long(), table),
                lambda: decode_attention(q, k, v, lens, table.long()),
                lambda: decode_attention(q, k, v, lens),
                lambda: decode_attention(q, k, v, lens[:1], table),
                lambda: decode_attention(q, k, v, lens, table[:1]),
                lambda: decode_attention(q, k, v, lens, table, k_new=q[:, :2]),
                lambda: decode_attention(q, k, v, lens, table, k_new=q, v_new=q),
                lambda: decode_attention(q, k, v, lens, table, out=q.float()),
                lambda: decode_attention(q, k, v, lens, table, out=q[:1].expand(2, -1, -1)),
                lambda: decode_attention(q, k[:1].expand(4, -1, -1, -1), v[:1].expand(4, -1, -1, -1), lens, table,
                                         k_new=q[:, :2], v_new=q[:, :2]),
                lambda: decode_attention(q.cpu(), k, v, lens, table),
                lambda: decode_attention(q, k, v, lens.cpu(), table),
                lambda: decode_attention(q.transpose(1, 2), k, v, lens, table),
                lambda: decode_attention(q, k, v, lens, table, window=1 << 40),
                lambda: decode_attention(q, k, v, lens, table, k_new=q[:, :2])):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros(2 * 4 * 64 + 1, dtype=torch.bfloat16, device=cuda_device)[1:].view(2, 4, 64)
    for bad in (lambda: decode_attention(odd, k, v, lens, table), lambda: decode_attention(q, k, v, lens, table, window=-1),
                lambda: decode_attention(q, k, v, lens, table, scale=float("nan")),
                lambda: decode_attention(q, k, v, lens, table, scale=1e60)):
        with pytest.raises(XlpkError) as e:
            bad()
        assert e.value.status == _abi.XLPK_ERR_INVALID_ARG
