"""The absorbed attention gives the same bits every time when partial scores take the exact exchange:
its buffer is handed between two SMs three times per key block, each time only once every thread
has what it read."""

import pytest
import torch

import latent_kv_cache_write_b200 as mla
from synth import configs as C

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wl", [C.WIDE_KEY, C.DECODE], ids=lambda w: w.name)
@pytest.mark.parametrize("n_keys", [79, 279])
def test_exact_exchange_repeats(cuda_ok, wl, n_keys):
    S = 300
    wl = wl.scaled(batch=1, n_heads=72, ring_slots=S, grid_h=1, grid_w=1)
    shape = mla.make_shape(wl)
    g = torch.Generator(device="cuda").manual_seed(3)
    # partial scores of some hundreds: past the bound of the rounded exchange
    q = (20 * torch.randn((1, 1, 72, wl.row_width), device="cuda", generator=g)).bfloat16()
    c = torch.randn((1, S, wl.row_width), device="cuda", generator=g).bfloat16()

    def run():
        o = torch.zeros((1, 1, 72, 512), device="cuda", dtype=torch.bfloat16)
        lse = torch.zeros((1, 1, 72), device="cuda")
        mla.mla_attend(shape, q, 1, n_keys - 1, c, 0, n_keys, 0.05, o, lse)
        assert mla.mla_device_error() == 0
        return o, lse

    o, lse = run()
    s = 0.05 * (q[0, 0].double() @ c[0, :n_keys].double().t())
    # the exchange is exact to float32 here, and the scores reach some hundreds
    assert ((lse[0, 0].double() - torch.logsumexp(s, 1)).abs() <= 1e-6 * s.abs().amax(1) + 2e-5).all()
    for _ in range(200):
        o2, lse2 = run()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
