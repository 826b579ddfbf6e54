"""The 4-bit KV cache on the GPU where values, memory and waits come to their ends."""
import pytest
import torch

from parity import compare_logits
from synthetic import make_prompt, make_weights
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
