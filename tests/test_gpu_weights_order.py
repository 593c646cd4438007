"""A handle used by the very next operation of its stream, on a B200.  The decodes' first kernels
load the packed weights before they wait for the kernel before them (programmatic launch), so
the packing has to be complete by then whatever its last kernel is: with fewer than 128 heads it is
the transpose that writes the weights the 8-bit decode loads."""
from __future__ import annotations

import pytest
import torch

from test_gpu_paged_q8 import DEV, Decode, gen, mla

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [1, 16, 64, 128])
def test_decode_directly_behind_the_packing_of_its_weights(H):
    D = Decode(H, 1, [70, 3], seed=91)
    kept, outs, wants = [D.w], [], []
    uks = [torch.randn(D.uk.shape, generator=gen(92 + i), device=DEV).to(torch.bfloat16) / 16 for i in range(6)]
    bufs = [torch.empty(2, 1, H, 128, dtype=torch.bfloat16, device=DEV) for _ in uks]
    torch.cuda.synchronize()
    for uk, out in zip(uks, bufs):           # nothing lies between packing and decode
        D.w = mla.mla_absorb_weights(D.d, uk, D.uv)
        kept.append(D.w)
        outs.append(D.run(out=out))
    torch.cuda.synchronize()
    for w in kept[1:]:
        D.w = w
        wants.append(D.run())
    assert mla.mla_get_device_error() == (0, 0)
    for o, w in zip(outs, wants):
        assert torch.equal(o, w)


def test_bf16_decode_directly_behind_the_packing_of_its_weights():
    H, B = 128, 3
    D = Decode(H, 1, [40], seed=93)          # its weights only
    g = gen(94)
    cache = (torch.randn(300, 576, generator=g, device=DEV) * 0.5).to(torch.bfloat16)
    offsets = torch.tensor([0, 100, 101, 300], dtype=torch.int32, device=DEV)
    qn = torch.randn(B, H, 128, generator=g, device=DEV).to(torch.bfloat16)
    qr = torch.randn(B, H, 64, generator=g, device=DEV).to(torch.bfloat16)
    ws = mla.workspace(mla.mla_decode_workspace_size(D.d, B))
    outs = [torch.empty(B, H, 128, dtype=torch.bfloat16, device=DEV) for _ in range(8)]
    uks = [torch.randn(D.uk.shape, generator=g, device=DEV).to(torch.bfloat16) / 16 for _ in range(4)]
    torch.cuda.synchronize()
    kept = []
    for uk, out in zip(uks, outs):
        kept.append(mla.mla_absorb_weights(D.d, uk, D.uv))
        mla.mla_decode_absorbed(D.d, kept[-1], cache, offsets, out, ws, q_nope=qn, q_rope=qr)
    torch.cuda.synchronize()
    for w, out, again in zip(kept, outs, outs[4:]):
        mla.mla_decode_absorbed(D.d, w, cache, offsets, again, ws, q_nope=qn, q_rope=qr)
        assert torch.equal(out, again)
    assert mla.mla_get_device_error() == (0, 0)


def test_append_directly_behind_a_kernel_that_writes_its_projection_weights():
    """mla_append_cache takes the caller's weights, which the operation before may have written."""
    n, dm = 8, 512
    g = gen(95)
    d = mla.make_dims(128, dm, 512, 64, 128, 128, "bf16")
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    h, new = rnd(n, dm), [(rnd(512, dm), rnd(64, dm)) for _ in range(6)]
    W1, W2 = torch.zeros(512, dm, dtype=torch.bfloat16, device=DEV), torch.zeros(64, dm, dtype=torch.bfloat16, device=DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    slot = torch.arange(n, dtype=torch.int64, device=DEV)
    got = [torch.zeros(n, 576, dtype=torch.bfloat16, device=DEV) for _ in new]
    torch.cuda.synchronize()
    for (a, b), cache in zip(new, got):
        W2.copy_(b)
        W1.copy_(a)
        mla.mla_append_cache(d, h, W1, W2, pos, slot, cache)
    torch.cuda.synchronize()
    for (a, b), cache in zip(new, got):
        want = torch.zeros_like(cache)
        mla.mla_append_cache(d, h, a, b, pos, slot, want)
        assert torch.equal(cache, want)
    assert mla.mla_get_device_error() == (0, 0)
