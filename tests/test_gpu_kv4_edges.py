"""The 4-bit KV cache on the GPU where values, memory and waits come to their ends."""
import os
import subprocess
import time

import pytest
import torch

import kv4_ref as ref
from parity import compare_logits
from synthetic import ModelConfig, make_prompt, make_weights
from test_gpu_kv4 import check, filled, gen
from test_gpu_kv4_decoder import GQA, forward, pm, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_prompt", [9, 10])
@pytest.mark.parametrize("block", [0, 4])
def test_v_rows_that_overflow_fp16_saturate_at_every_step(pm, block, n_prompt):
    """A V channel far beyond FP16's range is cached as 2,688, whichever way and at whichever step its row came."""
    cfg, w = GQA, make_weights(GQA, 5, device="cuda")
    d, G, hd = 21, cfg.n_heads // cfg.n_kv_heads, cfg.head_dim
    w["wv"][:, d] = w["wv"][:, d].sign() * 60000
    for h in range(G):                                    # what the first KV head's channel d does to the residual
        w["wo"][:, :, h * hd + d] /= 256
    prompt, force = make_prompt(cfg.vocab, n_prompt, 6), make_prompt(cfg.vocab, 8, 7)
    with pm.Decoder(cfg, w, 64, prefill_block=block, kv4=True) as dec:
        _, lg = run(dec, cfg, prompt, force)
    want = forward(cfg, w, torch.cat((prompt, force[:-1])).long().cuda())[n_prompt - 1:]
    compare_logits(lg.cpu(), want.cpu())


def _busy(stream, seconds=0.03):
    """Work that keeps the stream for about that long."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(seconds * 1.9e9))


def _reuse(shape, dtype):
    """What the allocator gives the current stream next for this shape, overwritten."""
    return [torch.full(shape, 7.0, dtype=dtype, device="cuda") for _ in range(8)]


@pytest.mark.parametrize("n", [1, 300])
def test_temporaries_passed_to_another_stream(pm, n):
    """Inputs and outputs that the caller lets go of while the stream has yet to come to them."""
    g = torch.Generator("cuda").manual_seed(n)
    k, v, q = (torch.randn(n, h, 128, generator=g, device="cuda").half() for h in (2, 2, 8))
    want = pm.KV4Cache(2, 128, 400)
    want.append(k, v, 5)
    out, rows = want.attend(q, 5), want.read(5, n)
    cache, s = pm.KV4Cache(2, 128, 400), torch.cuda.Stream()
    for _ in range(3):
        a, b, c, o, r = k.clone(), v.clone(), q.clone(), torch.empty_like(q), (torch.empty_like(k), torch.empty_like(v))
        s.wait_stream(torch.cuda.current_stream())
        _busy(s)
        cache.append(a, b, 5, stream=s)
        got = cache.attend(c, 5, stream=s)
        cache.attend(c, 5, out=o, stream=s)
        cache.read(5, n, out=r, stream=s)
        taken = {t.data_ptr() for t in (a, b, c, o, *r)}
        del a, b, c, o, r
        fresh = [t for x in (k, q) for t in _reuse(x.shape, x.dtype)]
        assert not taken & {t.data_ptr() for t in fresh}
        torch.cuda.synchronize()
        assert torch.equal(got, out) and all((t == 7).all() for t in fresh)
        assert torch.equal(cache.k_codes, want.k_codes) and torch.equal(cache.v_scales, want.v_scales)
        assert all(torch.equal(x, y) for x, y in zip(cache.read(5, n), rows))


def test_a_cache_let_go_of_while_another_stream_has_yet_to_read_it(pm):
    g = torch.Generator("cuda").manual_seed(1)
    k, q = (torch.randn(300, h, 128, generator=g, device="cuda").half() for h in (2, 8))
    cache, s = pm.KV4Cache(2, 128, 400), torch.cuda.Stream()
    cache.append(k, k, 0)
    want = cache.attend(q, 0)
    s.wait_stream(torch.cuda.current_stream())
    _busy(s)
    got = cache.attend(q, 0, stream=s)
    places, shapes = {t.data_ptr() for t in (cache.k_codes, cache.v_scales)}, (cache.k_codes.shape, cache.v_scales.shape)
    del cache
    fresh = [t for shape in shapes for t in _reuse(shape, torch.uint8)]
    assert not places & {t.data_ptr() for t in fresh}
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_the_caches_tensors_are_read_where_they_are(pm):
    """Another memory under a tensor of the cache is used, another size refused, another tensor in its place too."""
    g = torch.Generator("cuda").manual_seed(2)
    k, q = (torch.randn(30, h, 64, generator=g, device="cuda").half() for h in (2, 4))
    cache, other = pm.KV4Cache(2, 64, 40), pm.KV4Cache(2, 64, 40)
    cache.append(k, -k, 3)
    want = cache.attend(q, 3)
    names = ("k_codes", "k_scales", "v_codes", "v_scales")
    for name in names:
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(other, name))
        moved = getattr(cache, name).clone()
        getattr(cache, name).fill_(0x11)                  # (what a stale address would read)
        getattr(cache, name).set_(moved)
    assert torch.equal(cache.attend(q, 3), want)
    cache.append(-k, k, 3)
    other.append(-k, k, 3)
    assert all(torch.equal(getattr(cache, n)[:, 3:33], getattr(other, n)[:, 3:33]) for n in names)
    for name, change in (("v_scales", lambda t: t.resize_(2, 80, 4)), ("k_codes", lambda t: t.set_(t[:, :20]))):
        cache = pm.KV4Cache(2, 64, 40)
        change(getattr(cache, name))
        for call in (lambda: cache.append(k, k, 3), lambda: cache.read(3, 2), lambda: cache.attend(q, 3),
                     lambda: cache.attend(q, 3, stream=torch.cuda.Stream())):
            with pytest.raises(ValueError, match="no longer"):
                call()


def test_a_scale_that_32_bits_cannot_hold(pm):
    """One that vanishes in FP32 would be taken for 0, which selects 1 / sqrt(head_dim)."""
    cache = pm.KV4Cache(2, 64, 40)
    q = torch.randn(3, 4, 64, device="cuda").half()
    cache.append(q[:, :2], q[:, 2:], 0)
    for scale in (1e-60, -1e-60, 2.0 ** -150, 1e39):
        with pytest.raises((ValueError, pm.LFError)):
            cache.attend(q, 0, scale=scale)
    # the smallest that it can hold leaves every score at 0: the mean of what a row sees
    v = cache.read(0, 3, torch.float32)[1]
    mean = (v.cumsum(0) / torch.arange(1, 4, device="cuda")[:, None, None]).repeat_interleave(2, 1)
    assert torch.allclose(cache.attend(q, 0, scale=2.0 ** -149).float(), mean, rtol=2.0 ** -10, atol=2.0 ** -20)
    assert torch.equal(cache.attend(q, 0, scale=0.0), cache.attend(q, 0, scale=0.125))


WIDE8 = ModelConfig("wide8", 2, 512, 8, 1, 64, 512, 777)


@pytest.mark.parametrize("cfg,n", [(GQA, 600), (WIDE8, 333), (GQA, 1500)])
def test_a_wait_of_the_batched_prefills_attention_that_runs_out(pm, cfg, n):
    """A hand-over that never comes (test hook): the kernels end by themselves, the handle says so, and the same
    kernels are right in the next handle."""
    w, prompt, force = make_weights(cfg, 5, device="cuda"), make_prompt(cfg.vocab, n, 6), make_prompt(cfg.vocab, 4, 7)
    with pm.Decoder(cfg, w, n + 4, prefill_block=n, kv4=True, fault_step=pm.FAULT_PREFILL) as dec:
        dec.prefill(prompt.cuda())
        assert dec.sync() == 6
        with pytest.raises(pm.LFError, match="STATE"):
            dec.decode(1)
    with pm.Decoder(cfg, w, n + 4, prefill_block=n, kv4=True) as dec:
        _, lg = run(dec, cfg, prompt, force)
    want = forward(cfg, w, torch.cat((prompt, force[:-1])).long().cuda())[n - 1:]
    compare_logits(lg.cpu(), want.cpu())


def test_the_wait_limit_of_a_handle_bounds_its_prefills_attention(pm):
    """wait_timeout_ns = 20 ms over three layers; the default would take 2 s for each."""
    cfg, n = GQA, 600
    w, prompt = make_weights(cfg, 5, device="cuda"), make_prompt(cfg.vocab, n, 6).cuda()
    with pm.Decoder(cfg, w, n + 4, prefill_block=n, kv4=True, fault_step=pm.FAULT_PREFILL, wait_timeout_ns=20_000_000) as dec:
        start = time.monotonic()
        dec.prefill(prompt)
        assert dec.sync() == 6
        assert 0.02 < time.monotonic() - start < 2.0


def test_a_handles_error_is_its_own(pm):
    """A wait that ran out in one handle neither latches in another, nor is lost to whoever asks first, nor outlives
    lf_reset."""
    cfg, n = GQA, 600
    w, prompt, force = make_weights(cfg, 5, device="cuda"), make_prompt(cfg.vocab, n, 6), make_prompt(cfg.vocab, 4, 7)
    cache = pm.KV4Cache(2, 64, 32)
    with pm.Decoder(cfg, w, n + 4, prefill_block=n, kv4=True, fault_step=pm.FAULT_PREFILL, wait_timeout_ns=20_000_000) as a, \
            pm.Decoder(cfg, w, n + 4, prefill_block=n, kv4=True) as b:
        a.prefill(prompt.cuda())
        torch.cuda.synchronize()
        assert cache.sync() == 0
        _, lg = run(b, cfg, prompt, force)                # b.sync() is 0
        assert a.sync() == 6
        b.reset()
        _, again = run(b, cfg, prompt, force)
        assert a.sync() == 6 and torch.equal(lg, again)
        a.reset()
        assert a.sync() == 0
        # one that nobody asked for before the reset
        a.prefill(prompt.cuda())
        a.reset()
        assert a.sync() == 0 and cache.sync() == 0


def test_waits_that_run_out_outside_a_handle(pm, tmp_path):
    """kv4_expiry.cu, in a process of its own: every type and head size, tiles of their own and shared ones."""
    from persistent_monokernel_gb300 import build
    here, exe = os.path.dirname(os.path.abspath(__file__)), str(tmp_path / "kv4_expiry")
    objs = [os.path.join(build.BUILD, f) for f in ("lf_kv4.o", "lf_kv4_tc.o")]
    if not all(os.path.exists(o) for o in objs):
        build.build(force=True)
    subprocess.run([build.nvcc(), *build.ARCH, "-O1", "-std=c++17", os.path.join(here, "kv4_expiry.cu"), *objs, "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


def test_no_gradient_is_dropped_in_silence(pm):
    cache = pm.KV4Cache(2, 64, 40)
    q, k, out = (torch.randn(5, h, 64, device="cuda").half() for h in (4, 2, 4))
    cache.append(k, k, 0)
    want = cache.attend(q, 0)
    rows = cache.read(0, 5)
    leaf, kl = q.clone().requires_grad_(), k.clone().requires_grad_()
    for call in (lambda: cache.attend(leaf, 0), lambda: cache.attend(leaf * 2, 0), lambda: cache.attend(q, 0, out=leaf),
                 lambda: cache.append(kl, k, 0), lambda: cache.append(k, kl, 0), lambda: cache.read(0, 5, out=(kl, k)),
                 lambda: cache.attend(leaf, 0, stream=torch.cuda.Stream())):
        with pytest.raises(ValueError, match="gradient"):
            call()
    assert torch.equal(cache.attend(leaf.detach(), 0), want)
    for off in (torch.no_grad(), torch.inference_mode()):
        with off:
            cache.append(kl, kl, 0)
            assert torch.equal(cache.attend(leaf, 0, out=out), want)
            assert all(torch.equal(a, b) for a, b in zip(cache.read(0, 5), rows))


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_row_offsets_of_one_head_past_31_bits(pm, dtype):
    """One head of 33.6 million positions: its last rows' codes lie past 2^31 bytes from the head's first."""
    hd, cap, n, heads = 128, (1 << 25) + 4096, 300, 8
    cache = pm.KV4Cache(1, hd, cap)
    assert (cap - n) * (hd // 2) > 1 << 31
    g = torch.Generator("cuda").manual_seed(5)
    k, v = (torch.randn(n, 1, hd, generator=g, device="cuda").to(dtype) for _ in range(2))
    cache.append(k, v, cap - n)
    want = [ref.values(*ref.quantise(t)) for t in (k, v)]
    assert all(torch.equal(a.double(), b) for a, b in zip(cache.read(cap - n, n, dtype), want))
    kk, vv = (t.transpose(0, 1) for t in want)
    for rows in (1, 5, 150):
        q = torch.randn(rows, heads, hd, generator=g, device="cuda").to(dtype)
        # the window covers just what was written: the reference's position 0 is the cache's cap - n
        w = n - rows + 1
        check(cache.attend(q, cap - rows, window=w), *ref.attention(q, kk, vv, n - rows, n, w, 0))
    assert cache.sync() == 0


def test_sync_inside_a_capture_is_refused_and_the_capture_goes_on(pm):
    cache = pm.KV4Cache(2, 64, 40)
    q = torch.randn(3, 4, 64, device="cuda").half()
    cache.append(q[:, :2], q[:, 2:], 0)
    want = cache.attend(q, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cache.attend(q, 0)
        assert cache.sync() == 7                          # LF_ERR_NOT_SUPPORTED
        cache.append(q[:, :2], q[:, 2:], 0)
    graph.replay()
    assert cache.sync() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n,good", [(2, 1), (8, 3), (40, 17), (700, 333)])
def test_positions_never_written_do_not_reach_rows_that_do_not_see_them(pm, dtype, hd, n, good):
    """A block padded behind its first rows: the padded rows see positions that hold whatever the memory held, among
    it scales that stand for NaN."""
    pos = 600
    cache, (k, v) = filled(pm, 2, hd, pos + n + 3, hd + n)
    q = torch.randn(n, 16, hd, generator=gen(n), device="cuda").to(dtype)
    want, bound = ref.attention(q[:good], k, v, pos, pos + good, 0, 0)
    for byte in (0x7f, 0xff):
        for s in (cache.k_scales, cache.v_scales):
            s[:, pos + good:] = byte
        check(cache.attend(q, pos)[:good], want, bound)
        check(cache.attend(q[:good], pos), want, bound)


def test_a_stream_of_another_library_may_end_before_the_tensors(pm):
    """Nothing of the allocator's holds on to an ExternalStream when the memory is let go of."""
    import ctypes
    rt, handle = torch.cuda.cudart(), ctypes.c_void_p()
    assert int(rt.cudaStreamCreate(ctypes.addressof(handle))) == 0
    cache = pm.KV4Cache(2, 128, 400)
    k, q = (torch.randn(300, h, 128, generator=gen(h), device="cuda").half() for h in (2, 8))
    torch.cuda.synchronize()
    s = torch.cuda.ExternalStream(handle.value)
    cache.append(k, k, 0, stream=s)
    out = torch.empty_like(q)
    cache.attend(q, 0, out=out, stream=s)
    s.synchronize()
    want = cache.attend(q, 0)
    assert torch.equal(out, want)
    # (what the allocator made for the call itself, on s, goes back before s does)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    assert int(rt.cudaStreamDestroy(handle.value)) == 0
    del cache, k, q, out
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    assert torch.ones(1 << 20, device="cuda").sum() == 1 << 20
