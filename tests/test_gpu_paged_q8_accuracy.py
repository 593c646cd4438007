"""The 8-bit paged decode where its probabilities are hardest to hold, on a B200, against a plain
computation in 64 bits: a few tokens that take most of the softmax's weight and carry little
value (attention sinks) over a background that makes up the output.

Tolerance: the library's bf16 tolerance (helpers.assert_close, 2e-2 of the RMS of a head's 128
outputs).  A probability leaves as three terms of 3 significant bits, each within half a step
(2^-3) of what the terms before it left, so it is within 2^-9 of itself however small its share of
the softmax is (down to 2^-18 of the row's largest, 12.5 nats; the least step is 2^-27 of that).  An output that weighs
values of one sign is then within 2^-9 of itself, the partial's fp16 adds 2^-11, the output's own
rounding 2^-8: 0.0064 |y|, and the largest of 128 outputs is about 3 RMS (0.019)."""
from __future__ import annotations

import pytest
import torch

from helpers import assert_close
from test_gpu_paged_q8 import DC, DEV, DR, E4M3, PAGE, ROW, SCALE, Decode, gen, mla

pytestmark = pytest.mark.gpu


def set_scores(D, nats, small, noise=0.0, seed=5, level=1.0 / 16):
    """The rows of sequence 0: token i's score is nats[i] for every head (rotary column 0, which
    every query reads with weight 1 / SCALE) plus what q_nope makes of the latents, times
    `noise`; latents are a common mean plus a spread, zero where `small`."""
    n = len(nats)
    g = gen(seed)
    rows = torch.zeros(n, ROW, device=DEV)
    rows[:, :DC] = torch.randn(DC, generator=g, device=DEV) * 0.5 + torch.randn(n, DC, generator=g, device=DEV) * 0.3
    rows[small, :DC] = 0
    rows[:, DC] = nats
    pos = torch.arange(n, device=DEV)
    D.codes[D.table[0].long()[pos // PAGE], pos % PAGE] = (rows / level).to(E4M3).view(torch.uint8)
    D.scales[:] = level
    D.qn.mul_(noise)
    D.qr.zero_()
    D.qr[..., 0] = 1 / SCALE


def none_of(n):
    return torch.zeros(n, dtype=torch.bool, device=DEV)


@pytest.mark.parametrize("H,Q", [(16, 1), (32, 1), (128, 1), (128, 2), (24, 4)])
@pytest.mark.parametrize("nats", [5.0, 7.0, 10.0, 12.0])
@pytest.mark.parametrize("n", [128, 100])
def test_one_sink_of_little_value(H, Q, nats, n):
    D = Decode(H, Q, [n], seed=71)
    at = torch.arange(n, device=DEV) == 0
    set_scores(D, nats * at.float(), at)
    D.check(f"H={H} q_len={Q} one sink {nats} nats, {n} tokens")


@pytest.mark.parametrize("H", [16, 32, 128])
@pytest.mark.parametrize("valued", [False, True])
@pytest.mark.parametrize("nats,first,every", [(7.0, 3.5, 128), (7.25, 3.5, 128), (7.5, 3.5, 128), (5.5, 3.0, 128),
                                              (8.0, 2.0, 120), (10.0, 3.0, 128), (9.0, 3.0, 64)])
def test_sinks_in_every_tile(H, valued, nats, first, every):
    """The first sink sets the reference of the probabilities, the later ones are below it by
    `first` nats, and the background by `nats` more."""
    n = 4096
    D = Decode(H, 1, [n], seed=72)
    i = torch.arange(n, device=DEV)
    at = i % every == 0
    set_scores(D, nats * at.float() + first * (i == 0), none_of(n) if valued else at)
    D.check(f"H={H} sinks {nats} + {first} nats every {every}, valued={valued}")


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("sigma", [0.3, 2.0, 4.0])
@pytest.mark.parametrize("peak", [0.0, 8.0])
def test_spread_scores(H, sigma, peak):
    """Scores of a spread of some nats, alone and under peaks every 120 tokens."""
    n = 3000
    D = Decode(H, 1, [n], seed=73)
    i = torch.arange(n, device=DEV)
    at = i % 120 == 0
    set_scores(D, peak * at.float() + sigma * torch.randn(n, generator=gen(9), device=DEV), at, noise=0.2)
    D.check(f"H={H} sigma {sigma} nats, peaks of {peak}")


# Pages of one sequence whose scales differ, as appends make them: a page of zeros gets the scale 1,
# one large value raises its whole page's.  The formula weighs each value by its own page's scale, so
# every page's share of the output has to keep its precision beside any other's scale.

def filled(H, Q, rows, seed, qgain, dead_column=None):
    """A decode over one sequence whose pages mla_append_paged_q8 made from rows [n, 576]."""
    n = len(rows)
    D = Decode(H, Q, [n], seed=seed, qgain=qgain)
    if dead_column is not None:              # a latent that neither scores nor outputs use
        D.uk[..., dead_column] = 0
        D.uv[..., dead_column] = 0
        D.w = mla.mla_absorb_weights(D.d, D.uk, D.uv)
    rows = rows.to(torch.bfloat16)
    zero = torch.zeros(n, DR, dtype=torch.bfloat16, device=DEV)
    mla.mla_append_paged_q8(D.d, rows[:, :DC].contiguous(), zero, torch.tensor([0, n], dtype=torch.int32, device=DEV),
                            D.lens, D.codes, D.scales, D.table)
    return D


@pytest.mark.parametrize("H,Q", [(16, 1), (128, 1), (24, 3)])
@pytest.mark.parametrize("size", [0.1, 1e-2, 1e-3, 1e-6, 1e-15])
@pytest.mark.parametrize("zeros", ["first page", "second page", "first tile", "every other", "last"])
def test_pages_of_zeros_beside_small_latents(H, Q, size, zeros):
    n, g = 700, gen(81)
    mean = torch.randn(ROW, generator=g, device=DEV)
    rows = size * (mean + 0.5 * torch.randn(n, ROW, generator=g, device=DEV))
    page = torch.arange(n, device=DEV) // PAGE
    rows[{"first page": page == 0, "second page": page == 1, "first tile": page < 2, "every other": page % 2 == 0,
          "last": page == (n - 1) // PAGE}[zeros]] = 0
    D = filled(H, Q, rows, 82, min(0.3 / size, 1e15))
    assert float(D.scales[D.table[0].long()].amax()) == 1.0
    D.check(f"H={H} q_len={Q} zeros: {zeros}, others {size}")


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("ratio", [2 ** 5, 2 ** 8, 2 ** 10, 2 ** 12, 2 ** 20])
@pytest.mark.parametrize("where", ["every other", "first", "last"])
def test_a_large_value_in_some_pages(H, ratio, where):
    n, g = 1000, gen(83)
    rows = torch.randn(ROW, generator=g, device=DEV) + 0.5 * torch.randn(n, ROW, generator=g, device=DEV)
    page = torch.arange(n, device=DEV) // PAGE
    hit = {"every other": page % 2 == 1, "first": page == 0, "last": page == (n - 1) // PAGE}[where]
    rows[hit & (torch.arange(n, device=DEV) % PAGE == 7), 5] = 3.0 * ratio
    filled(H, 1, rows, 84, 0.3, dead_column=5).check(f"H={H} ratio {ratio} {where}")


@pytest.mark.parametrize("H,Q", [(16, 1), (128, 1), (64, 3)])
@pytest.mark.parametrize("exps", [(0, 25), (-30, 30, 0), (5, 0, 0, -5, -11, -11), (0, 0, 0, -60), (0.4, 5.3), (4, 0), (0, 5)])
def test_scales_of_any_ratio(H, Q, exps):
    """Full-range pages times any scales: those of the largest make up the output."""
    lens = [1200, 64, 130, 65, 128]
    Decode(H, Q, lens, seed=85, exps=exps, qgain=2.0 ** -max(max(exps), 0)).check(f"H={H} q_len={Q} exps={exps}")


def test_nan_behind_the_end_of_a_tile_of_two_scales():
    for n in (100, 65, 64):
        D = Decode(32, 1, [n], seed=86, exps=(0, 9), qgain=2.0 ** -9)
        want = D.check(f"{n} tokens")
        last = int(D.table[0, (n - 1) // PAGE])
        if n % PAGE:
            D.codes[last, n % PAGE:] = 0xFF
        assert torch.equal(D.check(f"{n} tokens, NaN behind them"), want)


def test_bad_page_beside_a_page_of_another_scale():
    D = Decode(16, 1, [500], seed=87, exps=(0, 12, -3), qgain=2.0 ** -12)
    keep = int(D.table[0, 3])
    D.table[0, 3] = -1
    out = D.run()
    assert mla.mla_get_device_error()[0] == mla.MLA_ERR_OUT_OF_RANGE
    D.table[0, 3] = keep
    D.codes[keep] = 0
    assert_close(out.float(), D.plain(), "bf16", "bad page")
