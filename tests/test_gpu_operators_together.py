"""The stand-alone operators used as one: a sampler on top of the decode forks its
sequences by their alternatives, decodes on, scores what came out, and gives pages back."""
import math

import pytest
import torch

import synth
from persistent_decode_b200 import decode_attention, token_logprobs, workload

from tests.gpu_util import oracle_for

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_beam_search_over_the_paged_decode(cuda_device):
    # the best `B` continuations, found by fork + reserve + decode; each beam's own tokens,
    # decoded again from the prompt in a contiguous cache, must give the same log probabilities
    B, steps = 4, 6
    cfg = synth.get_config("tiny", batch=B, steps=steps + 2, kv_len=125)
    m = workload.build(cfg, device=cuda_device, norm_std=0.1, paged=True, same_prompt=True, spare_pages=2 * B)
    lens = torch.full((B,), cfg.kv_len, dtype=torch.int32, device=cuda_device)
    pool = m.engine.page_pool(lens)
    beams = [[] for _ in range(B)]
    scores = torch.tensor([0.0] + [-math.inf] * (B - 1), dtype=torch.float64)
    logits = torch.empty(1, B, cfg.vocab, dtype=torch.float32, device=cuda_device)
    out = torch.empty(1, B, dtype=torch.int32, device=cuda_device)
    m.engine.set_state(m.start_tokens.tolist(), [cfg.kv_len] * B)
    for s in range(steps):
        pool.reserve(pool.seq_lens + 1)
        m.engine.decode(1, out, logits=logits)
        m.engine.check()
        pool.seq_lens += 1
        r = token_logprobs(logits[0], out[0], top_k=B)
        assert torch.equal(r.top_ids[:, 0], out[0]) and int(r.rank.max()) == 0     # the greedy token leads
        total = (scores[:, None] + r.top_logprobs.double().cpu()).reshape(-1)
        best = torch.sort(total, descending=True, stable=True).indices[:B].tolist()
        parents, toks = [i // B for i in best], [int(r.top_ids[i // B, i % B]) for i in best]
        scores = total[best]
        beams = [beams[p] + [t] for p, t in zip(parents, toks)]
        pool.fork(_i32(parents))
        if s % 3 == 2:
            pool.compact()
        pool.check()
        m.engine.set_state(toks, pool.seq_lens.tolist())
    flat = workload.build(cfg, device=cuda_device, norm_std=0.1, weights=m.weights, same_prompt=True)
    workload.reset_state(flat)
    scored = flat.engine.score(_i32(beams).t().contiguous(), top_k=1)
    flat.engine.check()
    # the same arithmetic on the same values: the forked, compacted cache decodes to the same bits
    want = scored.logprob.double().cpu().sum(0)
    assert torch.allclose(want, scores, rtol=1e-6, atol=0)
    assert len({tuple(b) for b in beams}) == B


def test_score_matches_the_oracle(cuda_device):
    cfg = synth.get_config("tiny", batch=2, steps=9)
    m = workload.build(cfg, device=cuda_device, norm_std=0.1)
    g = torch.Generator().manual_seed(3)
    toks = torch.randint(0, cfg.vocab, (7, 2), generator=g, dtype=torch.int32)
    workload.reset_state(m)
    r = m.engine.score(toks.to(cuda_device), top_k=3)
    m.engine.check()
    o = oracle_for(m)
    inp = m.start_tokens.tolist()
    for s in range(7):
        lg, _ = o.step(inp)
        lp = torch.log_softmax(lg.double(), 1)
        for b in range(2):
            # logits agree to 1e-2 in relative norm; that is their bound on a log probability too
            assert abs(float(r.logprob[s, b]) - float(lp[b, toks[s, b]])) <= 2e-2 * float(lg[b].abs().max())
        inp = toks[s].tolist()
    empty = m.engine.score(toks[:0].to(cuda_device))
    assert empty.logprob.shape == (0, 2)
    for bad in (toks.long().to(cuda_device), toks, toks[:, :1].to(cuda_device), toks[0].to(cuda_device)):
        with pytest.raises(ValueError):
            m.engine.score(bad)
    with pytest.raises(ValueError):     # a contiguous cache has no pages
        m.engine.page_pool(torch.zeros(2, dtype=torch.int32, device=cuda_device))


def test_score_in_parts_is_the_same(cuda_device, monkeypatch):
    cfg = synth.get_config("tiny", batch=2, steps=9)
    m = workload.build(cfg, device=cuda_device)
    toks = torch.randint(0, cfg.vocab, (7, 2), dtype=torch.int32, generator=torch.Generator().manual_seed(4)).to(cuda_device)
    whole = []
    for vocab_bytes in (28, 17):
        workload.reset_state(m)
        if vocab_bytes == 17:      # 131072 bytes: four steps at a time
            import persistent_decode_b200.engine as eng
            monkeypatch.setattr(eng, "SCORE_BYTES", 1 << 17)
        whole.append(m.engine.score(toks, top_k=2))
        m.engine.check()
    assert all(torch.equal(a, b) for a, b in zip(*whole))


def test_a_refused_score_moves_nothing(cuda_device, monkeypatch):
    import persistent_decode_b200.engine as eng
    from persistent_decode_b200 import XlpkError, _abi
    cfg = synth.get_config("tiny", batch=2, steps=9)
    m = workload.build(cfg, device=cuda_device)
    monkeypatch.setattr(eng, "SCORE_BYTES", 1 << 17)       # four steps at a time
    workload.reset_state(m)
    room = m.engine.max_seq - cfg.kv_len
    assert m.engine.room() == room
    g = torch.Generator().manual_seed(5)
    toks = torch.randint(0, cfg.vocab, (room + 1, 2), dtype=torch.int32, generator=g).to(cuda_device)
    want = m.engine.score(toks[:room], top_k=2)
    assert m.engine.room() == 0
    workload.reset_state(m)
    for n, k, status in ((room + 1, 2, _abi.XLPK_ERR_KV_FULL), (5, 65, _abi.XLPK_ERR_UNSUPPORTED), (5, -1, _abi.XLPK_ERR_INVALID_ARG),
                         (5, cfg.vocab + 1, _abi.XLPK_ERR_INVALID_ARG)):
        with pytest.raises(XlpkError) as e:
            m.engine.score(toks[:n], top_k=k)
        assert e.value.status == status
        assert m.engine.room() == room
    # positions and pending tokens are what they were: the same scores come out
    assert all(torch.equal(a, b) for a, b in zip(m.engine.score(toks[:room], top_k=2), want))
    m.engine.check()


def test_attention_reads_the_engines_cache(cuda_device):
    # the paged and the contiguous cache of the same model, bf16 and e4m3, after a decode
    for kv8 in (False, True):
        cfg = synth.get_config("tiny", batch=2, steps=5, kv_len=140)
        cfg = synth.fp8_kv(cfg) if kv8 else cfg
        paged = workload.build(cfg, device=cuda_device, paged=True)
        flat = workload.build(cfg, device=cuda_device, weights=paged.weights)
        out = torch.empty(5, 2, dtype=torch.int32, device=cuda_device)
        for m in (paged, flat):
            workload.reset_state(m)
            m.engine.decode(5, out)
            m.engine.check()
        q = torch.randn(2, cfg.n_q_heads, cfg.head_dim, device=cuda_device)
        lens = _i32([145, 91])
        scales = dict(k_scale=cfg.k_scale, v_scale=cfg.v_scale) if kv8 else {}
        for layer in range(cfg.n_layers):
            a = decode_attention(q, paged.k[layer], paged.v[layer], lens, paged.page_table, **scales)
            b = decode_attention(q, flat.k[layer], flat.v[layer], lens, **scales)
            assert torch.equal(a, b)
            k, v = (workload.kv_values(flat, w)[layer].double() for w in ("k", "v"))
            for i, n in enumerate([145, 91]):
                g = cfg.n_q_heads // cfg.n_kv_heads
                kk, vv = (t[i, :, :n].repeat_interleave(g, 0) for t in (k, v))
                s = torch.einsum("hd,htd->ht", q[i].double(), kk) / math.sqrt(cfg.head_dim)
                want = torch.einsum("ht,htd->hd", torch.softmax(s, 1), vv)
                assert float((a[i].double() - want).abs().max()) <= 2.0 ** -14 * float(vv.abs().max())


def test_a_window_lets_pages_go(cuda_device):
    # with the pages behind the window given back and the pool compacted, windowed attention reads the same
    cfg = synth.get_config("tiny", batch=2, steps=4, kv_len=700, prefill=False)
    m = workload.build(cfg, device=cuda_device, paged=True)
    lens = _i32([700, 420])
    q = torch.randn(2, cfg.n_q_heads, cfg.head_dim, device=cuda_device)
    kw = dict(window=200, sinks=3)
    want = [decode_attention(q, m.k[l], m.v[l], lens, m.page_table, **kw) for l in range(cfg.n_layers)]
    pool = m.engine.page_pool(lens)
    held = int((pool.refs > 0).sum())
    pool.trim(200, 3)
    pool.compact()
    pool.check()
    live = int((pool.refs > 0).sum())
    assert live < held and int(pool.page_table.max()) == live - 1
    for l in range(cfg.n_layers):
        m.k[l, live:] = float("nan")
        m.v[l, live:] = float("nan")
        assert torch.equal(decode_attention(q, m.k[l], m.v[l], lens, m.page_table, **kw), want[l])
