"""The paged appends at positions the caller gives, in every form of their kernels (16-byte rows and
any rows, bf16 and 8-bit pages), and over more sequences than a block has threads, on a B200.

Tolerances: as in test_gpu_paged_q8: a rotated key is rounded once to fp32 and once to bf16 (2^-8 of
itself + 2^-23 of the pair's size, and the fp64 angle of a position below 2^31 is off by 2^31 x 2^-53
x a few: nothing beside them); an 8-bit code is within half an E4M3 step of the exact value / scale."""
from __future__ import annotations

import pytest
import torch

from test_gpu_paged_q8 import DC, DEV, PAGE, ROW, append_inputs, code_values, dims, i32, mla, pow2_scale, rotate64

pytestmark = pytest.mark.gpu

NEW, PRE = [1, 70, 0, 200, 3], [0, 10, 64, 63, 127]


def positions(n, kind, g):
    if kind == "far":                        # unrelated, up to the largest
        pos = torch.randint(0, 2 ** 31 - 1, (n,), generator=g, device=DEV)
        pos[0], pos[-1] = 2 ** 31 - 1, 0
    elif kind == "same":
        pos = torch.full((n,), 4095, device=DEV)
    else:                                    # every other token, as where two sequences interleave, backwards
        pos = 2 * torch.arange(n, device=DEV).flip(0)
    return pos.to(torch.int32)


@pytest.mark.parametrize("kind", ["far", "same", "every other"])
@pytest.mark.parametrize("slack", [0, 8, 3])
def test_append_paged_at_given_positions(kind, slack):
    g, c, k, off, lens, table, pages, total = append_inputs(NEW, PRE, 61, slack=slack)
    pos = positions(len(c), kind, g)
    cache = torch.zeros(pages, PAGE, ROW, dtype=torch.bfloat16, device=DEV)
    mla.mla_append_paged(dims(), c, k, off, lens, cache, table, pos=pos)
    assert mla.mla_get_device_error() == (0, 0)
    want, at = rotate64(k, pos), 0
    for b, m in enumerate(NEW):
        place = torch.arange(PRE[b], total[b], device=DEV)
        got = cache[table[b].long()[place // PAGE], place % PAGE]
        w = want[at:at + m]
        pair = w.unflatten(1, (-1, 2)).norm(dim=-1).repeat_interleave(2, 1)
        assert torch.equal(got[:, :DC], c[at:at + m])
        assert ((got[:, DC:].double() - w).abs() <= 2.0 ** -8 * w.abs() + 2.0 ** -20 * pair).all()
        at += m


@pytest.mark.parametrize("kind", ["far", "same", "every other"])
@pytest.mark.parametrize("slack", [0, 8, 1])
def test_append_paged_q8_at_given_positions(kind, slack):
    g, c, k, off, lens, table, pages, total = append_inputs(NEW, [0] * 5, 62, slack=slack)
    pos = positions(len(c), kind, g)
    codes = torch.zeros(pages, PAGE, ROW, dtype=torch.uint8, device=DEV)
    scales = torch.full((pages,), float("nan"), device=DEV)
    mla.mla_append_paged_q8(dims(), c, k, off, lens, codes, scales, table, pos=pos)
    assert mla.mla_get_device_error() == (0, 0)
    x, at = torch.cat((c.double(), rotate64(k, pos)), 1), 0
    for b, m in enumerate(NEW):
        for a in range(0, m, PAGE):
            y, pg = x[at + a:at + min(m, a + PAGE)], int(table[b, a // PAGE])
            s = pow2_scale(float(y.abs().max().float()))
            assert float(scales[pg]) == s
            lim = torch.maximum(2.0 ** -4 * (y / s).abs(), torch.tensor(2.0 ** -10, device=DEV)) + 2.0 ** -20 * 448
            assert ((code_values(codes[pg, :len(y)]) - y / s).abs() <= lim).all()
        at += m


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B", [257, 1500])
def test_appends_of_many_sequences(q8, B):
    """One block looks through all sequences for its own: more of them than it has threads, some with
    nothing new."""
    new = [0 if i % 11 == 3 else 70 if i % 97 == 5 else 1 for i in range(B)]
    pre = [(37 * i) % 200 for i in range(B)]
    g, c, k, off, lens, table, pages, total = append_inputs(new, pre, 63)
    if q8:
        codes = torch.zeros(pages, PAGE, ROW, dtype=torch.uint8, device=DEV)
        scales = torch.full((pages,), 2.0 ** -60, device=DEV)
        mla.mla_append_paged_q8(dims(), c, k, off, lens, codes, scales, table)
        rows = code_values(codes) * scales.double()[:, None, None]
    else:
        cache = torch.zeros(pages, PAGE, ROW, dtype=torch.bfloat16, device=DEV)
        mla.mla_append_paged(dims(), c, k, off, lens, cache, table)
        rows = cache.double()
    assert mla.mla_get_device_error() == (0, 0)
    place = torch.cat([torch.arange(p, t, device=DEV) for p, t in zip(pre, total)])
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(new, device=DEV))
    pg = table.long()[seq, place // PAGE]
    got, want = rows[pg, place % PAGE], torch.cat((c.double(), rotate64(k, place)), 1)
    pair = torch.cat((c.double().abs(), want[:, DC:].unflatten(1, (-1, 2)).norm(dim=-1).repeat_interleave(2, 1)), 1)
    lim = 2.0 ** -8 * want.abs() + 2.0 ** -20 * pair
    if q8:
        lim = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * scales.double()[pg][:, None]) + 2.0 ** -20 * pair
    assert ((got - want).abs() <= lim).all()
    rows[pg, place % PAGE] = 0
    assert (rows == 0).all()                 # nothing else was written
