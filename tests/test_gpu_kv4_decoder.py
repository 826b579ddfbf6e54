"""The decoder on a 4-bit KV cache (lf_create_kv4) against a plain decoder in 64 bits whose K and V rows go through
the cache's format, at the logit tolerances of the other parity tests: a prefill as steps and batched, then decode
steps with forced tokens.

(The quantised values jump where a rounding is close to half-way; K and V are rounded to FP16 first on both sides, so
an FP32 difference moves a code only where it moves that rounding next to a border, which the tolerance covers: one
code of one row shifts a probability by a fraction of a percent.)"""
import math

import pytest
import torch

import kv4_ref as ref
from parity import compare_logits
from synthetic import ModelConfig, make_prompt, make_weights, make_weights_fp8, make_weights_mxfp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    import persistent_monokernel_gb300 as pm
    from persistent_monokernel_gb300 import build
    build.build()
    return pm


def forward(cfg, w, tokens, windows=None, quantised=True):
    """Logits of every position, FP64, all positions at once."""
    dev = w["embed"].device
    n, hd, G = len(tokens), cfg.head_dim, cfg.n_heads // cfg.n_kv_heads
    x = w["embed"][tokens].double()
    at = torch.arange(n, device=dev).double()
    ang = at[:, None] * cfg.rope_theta ** (-2.0 * torch.arange(hd // 2, device=dev).double() / hd)
    cos, sin = ang.cos(), ang.sin()

    def mat(name, l):
        m = w[name][l] if name != "lm_head" else w[name]
        if m.dtype == torch.uint8 and w[name + "_scale"].dtype == torch.float32:
            s = w[name + "_scale"][l] if name != "lm_head" else w[name + "_scale"]
            return ref.minifloat(m, 4, 3, 7) * s.double()[:, None]
        if m.dtype == torch.uint8:
            s = w[name + "_scale"][l] if name != "lm_head" else w[name + "_scale"]
            c = torch.stack((m & 15, m >> 4), -1).flatten(-2)
            return ref.e2m1(c) * torch.exp2(s.double() - 127).repeat_interleave(32, -1)
        return m.double()

    def norm(x, g):
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + cfg.rms_eps) * g.double()

    def rope(t):
        a, b = t[..., :hd // 2], t[..., hd // 2:]
        c, s = cos[:, None], sin[:, None]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    for l in range(cfg.n_layers):
        h = norm(x, w["attn_norm"][l])
        q = rope((h @ mat("wq", l).T).unflatten(-1, (-1, hd)))
        k = rope((h @ mat("wk", l).T).unflatten(-1, (-1, hd))).half()
        v = (h @ mat("wv", l).T).unflatten(-1, (-1, hd)).half()
        if quantised:
            k, v = (ref.values(*ref.quantise(t)) for t in (k, v))
        see = ref.seen(n, 0, n, windows[l] if windows else 0, dev)
        o = torch.empty(n, cfg.n_heads, hd, dtype=torch.float64, device=dev)
        for i in range(cfg.n_heads):
            s = (q[:, i] @ k[:, i // G].double().T / math.sqrt(hd)).masked_fill(~see, -math.inf)
            o[:, i] = torch.softmax(s, -1) @ v[:, i // G].double()
        x = x + o.flatten(1) @ mat("wo", l).T
        h = norm(x, w["ffn_norm"][l])
        if cfg.n_experts:
            r = h @ w["w_router"][l].double().T
            val, idx = r.topk(cfg.top_k_experts)
            gate = torch.softmax(val, -1)
            y = torch.zeros_like(x)
            for e in range(cfg.n_experts):
                rows, slot = (idx == e).nonzero(as_tuple=True)
                hh = h[rows]
                u = torch.nn.functional.silu(hh @ w["w_gate"][l, e].double().T) * (hh @ w["w_up"][l, e].double().T)
                y.index_add_(0, rows, gate[rows, slot, None] * (u @ w["w_down"][l, e].double().T))
            x = x + y
        else:
            x = x + (torch.nn.functional.silu(h @ mat("w_gate", l).T) * (h @ mat("w_up", l).T)) @ mat("w_down", l).T
    return norm(x, w["final_norm"]) @ mat("lm_head", 0).T


def run(dec, cfg, prompt, force):
    n = len(force)
    dec.prefill(prompt.cuda())
    lg = torch.empty((n, cfg.vocab), dtype=torch.float32, device="cuda")
    toks = dec.decode(n, debug_logits=lg, force_tokens=force.cuda())
    assert dec.sync() == 0
    return toks, lg


TINY = ModelConfig("tiny", 2, 256, 4, 4, 64, 1024, 4096)
GQA = ModelConfig("gqa", 3, 512, 8, 2, 128, 768, 1000)
WIDE = ModelConfig("wide", 2, 512, 8, 1, 64, 512, 777)
MOE = ModelConfig("moe", 2, 256, 4, 2, 64, 256, 600, n_experts=4, top_k_experts=2)


@pytest.mark.parametrize("block", [0, 16, 160])
@pytest.mark.parametrize("cfg,make,windows,n_prompt", [
    (TINY, make_weights, None, 64), (GQA, make_weights, None, 300), (GQA, make_weights, (0, 40, 7), 150),
    (WIDE, make_weights, None, 130), (MOE, make_weights, None, 90), (GQA, make_weights_fp8, None, 100),
    (TINY, make_weights_mxfp4, None, 70), (TINY, make_weights, (1, 1000), 1)])
def test_forced_decode_parity(pm, cfg, make, windows, n_prompt, block):
    w = make(cfg, 5, device="cuda")
    n = 12
    prompt, force = make_prompt(cfg.vocab, n_prompt, 6), make_prompt(cfg.vocab, n, 7)
    with pm.Decoder(cfg, w, n_prompt + n, layer_window=windows, prefill_block=block, kv4=True) as dec:
        toks, lg = run(dec, cfg, prompt, force)
        # the same sequence again on the same handle
        dec.reset()
        toks2, lg2 = run(dec, cfg, prompt, force)
    seq = torch.cat((prompt, force[:-1])).long().cuda()
    want = forward(cfg, w, seq, windows)[n_prompt - 1:]
    compare_logits(lg.cpu(), want.cpu())
    assert torch.equal(toks, toks2) and torch.equal(lg, lg2)
    top = want.topk(2).values
    sure = top[:, 0] - top[:, 1] > 0.05
    assert torch.equal(toks.long()[sure], want.argmax(-1)[sure])
    # and not the FP16 cache's logits: the 4-bit values are what is attended to
    if n_prompt > 60:
        plain = forward(cfg, w, seq, windows, quantised=False)[n_prompt - 1:]
        assert ((lg.double() - want).norm() < 0.1 * (plain - want).norm())


def test_prefill_then_generate_in_pieces(pm):
    """Chunks of a prompt, decode, more prompt, decode: the positions go on."""
    cfg, w = GQA, make_weights(GQA, 5, device="cuda")
    a, b = make_prompt(cfg.vocab, 50, 1), make_prompt(cfg.vocab, 45, 2)
    f, g = make_prompt(cfg.vocab, 5, 3), make_prompt(cfg.vocab, 4, 4)
    with pm.Decoder(cfg, w, 120, prefill_block=32, kv4=True) as dec:
        _, l1 = run(dec, cfg, a, f)
        # the last forced token is pending and runs as the next prefill's first position
        _, l2 = run(dec, cfg, b, g)
        info = dec.info()
    assert info["position"] == 50 - 1 + 5 + 1 + 45 - 1 + 4
    assert info["kv_cache_bytes"] == 2 * cfg.n_layers * 120 * cfg.kv_dim * 9 // 16
    seq = torch.cat((a, f, b, g[:-1])).long().cuda()
    want = forward(cfg, w, seq)
    compare_logits(l1.cpu(), want[49:54].cpu())
    compare_logits(l2.cpu(), want[99:103].cpu())


def test_generate_and_refusals(pm):
    cfg, w = TINY, make_weights(TINY, 5, device="cuda")
    prompt = make_prompt(cfg.vocab, 20, 6)
    with pm.Decoder(cfg, w, 64, kv4=True) as dec:
        out = dec.generate(prompt.numpy(), 10)
        dec.reset()
        assert (dec.generate(prompt.numpy(), 10) == out).all()
        for schedule in (pm.SCHED_GRID_BARRIER, pm.SCHED_MULTI_KERNEL):
            with pytest.raises(pm.LFError, match="NOT_SUPPORTED"):
                dec.set_schedule(schedule)
        with pytest.raises(pm.LFError, match="NOT_SUPPORTED"):
            dec.enable_trace(1)
        with pytest.raises(pm.LFError, match="CAPACITY"):
            dec.decode(100)


def test_the_fp16_cache_is_as_it_was(pm):
    """A 4-bit and an FP16 handle side by side: the FP16 one gives its own logits."""
    cfg, w = TINY, make_weights(TINY, 5, device="cuda")
    prompt, force = make_prompt(cfg.vocab, 40, 6), make_prompt(cfg.vocab, 8, 7)
    with pm.Decoder(cfg, w, 64) as a, pm.Decoder(cfg, w, 64, kv4=True) as b:
        _, la = run(a, cfg, prompt, force)
        _, lb = run(b, cfg, prompt, force)
        a.reset()
        _, lc = run(a, cfg, prompt, force)
    seq = torch.cat((prompt, force[:-1])).long().cuda()
    compare_logits(la.cpu(), forward(cfg, w, seq, quantised=False)[39:].cpu())
    assert torch.equal(la, lc) and not torch.equal(la, lb)
