"""The paged appends and the decode over the 8-bit paged cache, on a B200, against plain
computations in 64 bits.

Tolerances.  Appended rows: the latent's bits; a rotated key is rounded once to fp32 and once
to storage, so it is within (half a bf16 step = 2^-8 relative) + 2^-23 of the exact rotation,
fp32 storage within 2^-22.  Codes: within half an E4M3 step of value / scale, 2^-4 relative or,
where E4M3 is subnormal (step 2^-9), 2^-10 absolute, + 2^-22 for the fp32 quotient's input.
Decode: the library's bf16 tolerance (helpers.assert_close).  The kernel rounds queries to two
8-bit terms (at most 2^-8 relative, or 2^-17 of the row's largest value) and probabilities to three
(2^-9), which by the same count as bf16 operands (2^-8 each) is inside it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from helpers import assert_close

pytestmark = pytest.mark.gpu

mla = pytest.importorskip("compressed_kv_cache_absorbed_b200")

DEV = "cuda"
PAGE, ROW, DC, DR = 64, 576, 512, 64
E4M3 = torch.float8_e4m3fn
SCALE = 192 ** -0.5


def dims(H=128, dtype="bf16", **kw):
    d = dict(H=H, d_model=0, d_c=DC, d_hR=DR, qk_nope=128, v_head=128, dtype=dtype)
    d.update(kw)
    return mla.make_dims(**d)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def page_table(total, g, spare=3, width=None):
    blocks = [(n + PAGE - 1) // PAGE for n in total]
    pages = sum(blocks) + spare
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    t = torch.full((len(total), width or max(max(blocks), 1)), -7, dtype=torch.int32, device=DEV)
    at = 0
    for b, k in enumerate(blocks):
        t[b, :k] = perm[at:at + k]
        at += k
    return t, pages


def rotate64(k, pos, d_hR=DR):
    f = 10000.0 ** (-torch.arange(0, d_hR, 2, dtype=torch.float64, device=k.device) / d_hR)
    a = pos.double()[:, None] * f
    x, y = k.double()[:, 0::2], k.double()[:, 1::2]
    return torch.stack((x * a.cos() - y * a.sin(), x * a.sin() + y * a.cos()), -1).flatten(1)


def pow2_scale(amax):
    return max(2.0 ** -60, 2.0 ** int(np.ceil(np.log2(amax / 448)))) if amax > 0 else 1.0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def append_inputs(new, pre, seed, dt=torch.bfloat16, d_c=DC, d_hR=DR, slack=0):
    g = gen(seed)
    n = sum(new)
    kv = (torch.randn(n, d_c + d_hR + slack, generator=g, device=DEV)
          * torch.exp(0.7 * torch.randn(n, 1, generator=g, device=DEV))).to(dt)
    total = [a + k for a, k in zip(pre, new)]
    table, pages = page_table(total, g)
    off = i32([0] + list(np.cumsum(new)))
    return g, kv[:, :d_c], kv[:, d_c:d_c + d_hR], off, i32(total), table, pages, total


APPENDS = [([1], [0]), ([1] * 5, [0, 63, 64, 127, 300]), ([64, 0, 65, 1], [0, 64, 63, 5]),
           ([200, 3, 0, 129], [37, 0, 0, 64]), ([1000], [1])]


@pytest.mark.parametrize("slack", [0, 8, 3])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new,pre", APPENDS)
def test_append_paged_writes_the_rows(new, pre, dt, slack):
    g, c, k, off, lens, table, pages, total = append_inputs(new, pre, 5 + len(new), dt, slack=slack)
    cache = torch.randn(pages, PAGE, ROW, generator=g, device=DEV).to(dt)
    before = cache.clone()
    mla.mla_append_paged(dims(dtype=dt), c, k, off, lens, cache, table)
    assert mla.mla_get_device_error() == (0, 0)
    touched = torch.zeros(pages, PAGE, dtype=torch.bool, device=DEV)
    at = 0
    for b, m in enumerate(new):
        pos = torch.arange(pre[b], total[b], device=DEV)
        pg, row = table[b].long()[pos // PAGE], pos % PAGE
        got = cache[pg, row]
        assert torch.equal(got[:, :DC], c[at:at + m])
        want = rotate64(k[at:at + m], pos)
        rel = 2.0 ** -8 + 2.0 ** -23 if dt == torch.bfloat16 else 2.0 ** -22
        assert ((got[:, DC:].double() - want).abs() <= rel * want.abs() + 1e-30).all()
        touched[pg, row] = True
        at += m
    assert torch.equal(cache[~touched], before[~touched])


def test_append_paged_other_widths_and_given_positions():
    d = dims(H=4, d_c=32, d_hR=16, qk_nope=32, v_head=32, dtype="f32")
    new, pre = [3, 70], [10, 0]
    g, c, k, off, lens, table, pages, total = append_inputs(new, pre, 3, torch.float32, 32, 16)
    pos = i32([10 ** 8, 0, 12345678] + list(range(1000, 1070)))
    cache = torch.zeros(pages, PAGE, 48, device=DEV)
    mla.mla_append_paged(d, c, k, off, lens, cache, table, pos=pos)
    assert mla.mla_get_device_error() == (0, 0)
    want = rotate64(k, pos, 16)
    place = [(int(table[b, p // 64]), p % 64) for b in range(2) for p in range(pre[b], total[b])]
    got = torch.stack([cache[p, r] for p, r in place])
    assert torch.equal(got[:, :32], c)
    assert ((got[:, 32:].double() - want).abs() <= 2.0 ** -22 * want.abs().amax(1, keepdim=True)).all()
    assert int((cache != 0).any(-1).sum()) == len(place)


def code_values(codes):
    return codes.view(E4M3).double()


@pytest.mark.parametrize("slack", [0, 8, 1])
@pytest.mark.parametrize("gain", [1.0, 40.0, 1e-3])
@pytest.mark.parametrize("new,pre", APPENDS)
def test_append_paged_q8_codes_and_scales(new, pre, gain, slack):
    g, c, k, off, lens, table, pages, total = append_inputs(new, pre, 50 + len(new), slack=slack)
    old = torch.randn(pages, PAGE, ROW, generator=g, device=DEV) * gain
    scales = torch.tensor([pow2_scale(float(x)) for x in old.abs().amax((1, 2))], device=DEV)
    codes = (old / scales[:, None, None]).to(E4M3).view(torch.uint8)
    codes0, scales0 = codes.clone(), scales.clone()
    mla.mla_append_paged_q8(dims(), c, k, off, lens, codes, scales, table)
    assert mla.mla_get_device_error() == (0, 0)
    touched = torch.zeros(pages, PAGE, dtype=torch.bool, device=DEV)
    at = 0
    for b, m in enumerate(new):
        pos = torch.arange(pre[b], total[b], device=DEV)
        x = torch.cat((c[at:at + m].double(), rotate64(k[at:at + m], pos)), 1)
        for j in range(pre[b] // PAGE, (total[b] + PAGE - 1) // PAGE) if m else ():
            pg = int(table[b, j])
            a, e = max(pre[b], j * PAGE), min(total[b], (j + 1) * PAGE)
            y, held = x[a - pre[b]:e - pre[b]], a - j * PAGE
            s = pow2_scale(float(y.abs().max().float()))
            if held:
                s = max(s, float(scales0[pg]))
                ratio = float(scales0[pg]) / s
                again = (code_values(codes0[pg, :held]) * ratio).float().to(E4M3).view(torch.uint8)
                assert torch.equal(codes[pg, :held], again if ratio != 1 else codes0[pg, :held])
                touched[pg, :held] = True
            assert float(scales[pg]) == s
            got = code_values(codes[pg, held:held + len(y)])
            lim = torch.maximum(2.0 ** -4 * (y / s).abs(), torch.tensor(2.0 ** -10, device=DEV)) + 2.0 ** -22 * 448
            assert ((got - y / s).abs() <= lim).all()
            touched[pg, held:held + len(y)] = True
        at += m
    assert torch.equal(codes[~touched], codes0[~touched])
    idle = ~touched.any(1)
    assert torch.equal(scales[idle], scales0[idle])


def test_append_paged_q8_zero_rows_infinities_and_nan():
    c = torch.zeros(4, DC, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(4, DR, dtype=torch.bfloat16, device=DEV)
    c[1, 3], c[1, 4], c[1, 5] = float("inf"), float("-inf"), float("nan")
    c[2, 0] = 3.0e-30
    codes = torch.full((4, PAGE, ROW), 0x33, dtype=torch.uint8, device=DEV)
    scales = torch.full((4,), float("nan"), device=DEV)
    table = i32([[3], [1], [0], [2]])
    mla.mla_append_paged_q8(dims(), c, k, i32([0, 1, 2, 3, 4]), i32([1, 1, 1, 1]), codes, scales, table)
    assert mla.mla_get_device_error() == (0, 0)
    assert scales.tolist() == [2.0 ** -60, 1.0, 1.0, 1.0]    # pages of sequences 2, 1, 3, 0
    assert (codes[3, 0] == 0).all() and (codes[2, 0] == 0).all()
    assert [int(x) for x in codes[1, 0, 3:5]] == [0x7E, 0xFE] and int(codes[1, 0, 5]) & 0x7F == 0x7F
    assert (codes[:, 1:] == 0x33).all()


@pytest.mark.parametrize("q8", [False, True])
def test_append_reports_and_skips_what_is_out_of_range(q8):
    def run(off, lens, table, n=4):
        c = torch.ones(n, DC, dtype=torch.bfloat16, device=DEV)
        k = torch.zeros(n, DR, dtype=torch.bfloat16, device=DEV)
        if q8:
            codes = torch.zeros(3, PAGE, ROW, dtype=torch.uint8, device=DEV)
            mla.mla_append_paged_q8(dims(), c, k, i32(off), i32(lens), codes, torch.ones(3, device=DEV), i32(table))
        else:
            codes = torch.zeros(3, PAGE, ROW, dtype=torch.bfloat16, device=DEV)
            mla.mla_append_paged(dims(), c, k, i32(off), i32(lens), codes, i32(table))
        st, where = mla.mla_get_device_error()
        return st, where, (codes != 0).any(-1).sum(1).tolist()
    bad = mla.MLA_ERR_OUT_OF_RANGE
    assert run([0, 2, 4], [2, 2], [[0], [2]]) == (0, 0, [2, 0, 2])
    for off in ([1, 2, 4], [0, 3, 2], [0, 2, 3], [0, 5, 4], [0, -1, 4]):
        st, _, rows = run(off, [2, 2], [[0], [2]])
        assert st == bad and rows == [0, 0, 0], off
    assert run([0, 2, 4], [1, 2], [[0], [2]]) == (bad, 0, [0, 0, 2])      # fewer tokens than new ones
    assert run([0, 2, 4], [2, 65], [[0], [2]]) == (bad, 1, [2, 0, 0])     # more than the table's pages
    assert run([0, 2, 4], [2, 2], [[3], [2]]) == (bad, 0, [0, 0, 2])      # a page outside the cache
    assert run([0, 2, 4], [2, 2], [[-1], [2]]) == (bad, 0, [0, 0, 2])


# ------------------------------------------------------------------------- decode

def weights_of(H, seed):
    g = gen(seed)
    uk = (torch.randn(H, 128, DC, generator=g, device=DEV) / DC ** 0.5).to(torch.bfloat16)
    uv = (torch.randn(H, 128, DC, generator=g, device=DEV) / DC ** 0.5).to(torch.bfloat16)
    return uk, uv


def cache_of(pages, g, spread=0.3, exps=(0,)):
    x = torch.randn(pages, PAGE, ROW, generator=g, device=DEV) * 0.5
    x *= torch.exp(spread * torch.randn(pages, PAGE, 1, generator=g, device=DEV))
    s = torch.tensor([pow2_scale(float(v)) for v in x.abs().amax((1, 2))], device=DEV)
    codes = (x / s[:, None, None]).to(E4M3).view(torch.uint8)
    e = torch.tensor([exps[i % len(exps)] for i in range(pages)], device=DEV)
    return codes, s * torch.exp2(e.float())


def plain_decode(qn, qr, codes, scales, table, lens, uk, uv):
    """[B, q_len, H, 128] in 64 bits, sequence by sequence."""
    B, Q, H, _ = qn.shape
    out = torch.zeros(B, Q, H, 128, dtype=torch.float64, device=DEV)
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        pg = table[b, :(n + 63) // 64].long()
        rows = (code_values(codes[pg]) * scales[pg].double()[:, None, None]).reshape(-1, ROW)[:n]
        ql = torch.einsum("qhj,hjc->qhc", qn[b].double(), uk.double())
        z = SCALE * (torch.cat((ql, qr[b].double()), -1) @ rows.T)
        for t in range(Q):
            m = n - (Q - 1 - t)
            if m > 0:
                p = torch.softmax(z[t, :, :m], -1)
                out[b, t] = torch.einsum("hc,hvc->hv", p @ rows[:m, :DC], uv.double())
    return out


class Decode:
    def __init__(self, H, Q, lens, seed=1, exps=(0,), qgain=1.0, width=None):
        g = gen(seed)
        self.H, self.Q, self.B = H, Q, len(lens)
        self.table, pages = page_table([max(n, 0) for n in lens], g, width=width)
        self.codes, self.scales = cache_of(pages, g, exps=exps)
        self.lens = i32(lens)
        rnd = lambda w: torch.randn(self.B, Q, H, w, generator=g, device=DEV) * qgain  # noqa: E731
        self.qn, self.qr = rnd(128).to(torch.bfloat16), rnd(64).to(torch.bfloat16)
        self.uk, self.uv = weights_of(H, seed + 1)
        self.d = dims(H)
        self.w = mla.mla_absorb_weights(self.d, self.uk, self.uv)
        self.ws = self.workspace()

    def workspace(self):
        ws = mla.workspace(mla.mla_decode_q8_workspace_size(self.d, self.B, self.Q))
        return ws.fill_(0xFF)                # contents on entry do not matter: NaN patterns

    def run(self, out=None, ws=None):
        if out is None:
            out = torch.full((self.B, self.Q, self.H, 128), 3.0, dtype=torch.bfloat16, device=DEV)
        mla.mla_decode_absorbed_paged_q8(self.d, self.w, self.codes, self.scales, self.table, self.lens, out,
                                         self.ws if ws is None else ws, self.qn, self.qr)
        return out

    def plain(self):
        return plain_decode(self.qn, self.qr, self.codes, self.scales, self.table, self.lens, self.uk, self.uv)

    def check(self, what, out=None):
        got = self.run() if out is None else out
        assert mla.mla_get_device_error() == (0, 0)
        assert_close(got.float(), self.plain(), "bf16", what)
        return got


RAGGED = [0, 1, 63, 64, 65, 127, 128, 129, 300, 700]


@pytest.mark.parametrize("H", [1, 7, 16, 20, 32, 40, 64, 96, 100, 128])
@pytest.mark.parametrize("Q", [1, 2, 5])
def test_decode_heads_and_new_tokens(H, Q):
    Decode(H, Q, RAGGED, seed=H + Q).check(f"H={H} q_len={Q}")


@pytest.mark.parametrize("H,Q,lens", [(128, 1, [100]), (128, 1, [9000]), (16, 1, [20000, 1]), (64, 100, [333, 100, 40]),
                                      (3, 50, [500]), (128, 33, [64, 200]), (128, 1, [1] * 300), (64, 3, [517] * 40)])
def test_decode_lengths(H, Q, lens):
    Decode(H, Q, lens, seed=77).check(f"H={H} q_len={Q} B={len(lens)}")


@pytest.mark.parametrize("B", [1, 2, 3, 5, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("H", [16, 70, 128])
def test_decode_numbers_of_queries(H, B):
    """Rows of a merge CTA: one, a few (shared by warps), up to 16, up to 32, a rest; each with
    sequences of one piece and of many, and one without tokens."""
    lens = [3000 if i % 3 == 0 else 0 if i % 7 == 4 else 90 + i for i in range(B)]
    Decode(H, 1, lens, seed=B).check(f"H={H} B={B}")


@pytest.mark.parametrize("exps", [(0, 3, -4), (-40,), (40,), (0.37, -1.9), (0, 12)])
@pytest.mark.parametrize("H", [16, 128])
def test_decode_scales_of_the_pages(H, exps):
    # the scores grow with the scales: keep them in range so that the softmax is not one-hot
    gain = min(1.0, 2.0 ** -max(exps))
    Decode(H, 1, [700, 64, 130], seed=9, exps=exps, qgain=gain).check(f"H={H} exps={exps}")


@pytest.mark.parametrize("profile", ["sink", "growing", "falling", "spikes", "one_hot"])
@pytest.mark.parametrize("H", [16, 128])
def test_decode_uneven_scores(H, profile):
    """Scores that one token, a drift or rare tokens dominate: the running reference of the
    probabilities has to follow them up and down."""
    D = Decode(H, 1, [1500, 640], seed=21)
    for b in range(2):
        n = int(D.lens[b])
        pos = torch.arange(n, device=DEV)
        want = {"sink": 12.0 * (pos == 0), "growing": 30.0 * pos / n, "falling": 30.0 * (1 - pos / n),
                "spikes": 9.0 * (pos % 97 == 0), "one_hot": 80.0 * (pos == 517)}[profile].float()
        # rotary column 0 carries the profile; every head's query reads it with weight 1 / SCALE
        pg, row = D.table[b].long()[pos // PAGE], pos % PAGE
        s = D.scales[pg]
        full = code_values(D.codes[pg, row]).float() * s[:, None]
        full[:, DC] = want
        D.scales[pg] = torch.maximum(s, torch.full_like(s, 0.25))
        D.codes[pg, row] = (full / D.scales[pg][:, None]).to(E4M3).view(torch.uint8)
    D.qr[..., 0] = 1 / SCALE
    D.check(f"H={H} {profile}")


def test_what_lies_behind_a_sequence_does_not_matter():
    D = Decode(64, 2, [100, 1, 65, 200], seed=31)
    want = D.check("before")
    for b, n in enumerate([100, 1, 65, 200]):
        if n % PAGE:
            D.codes[int(D.table[b, n // PAGE]), n % PAGE:] = 0x7F        # NaN codes
    assert torch.equal(D.check("NaN behind the end"), want)


def test_nan_in_a_row_that_counts_reaches_its_sequence_only():
    D = Decode(16, 1, [100, 90], seed=32)
    D.codes[int(D.table[0, 0]), 5, 7] = 0x7F
    out = D.run()
    assert mla.mla_get_device_error() == (0, 0)
    assert torch.isnan(out[0]).all()
    assert_close(out[1].float(), D.plain()[1], "bf16", "the other sequence")


def test_bad_lengths_and_pages_are_reported():
    D = Decode(128, 1, [130, 300, 64], seed=33)
    good = D.run()
    D.lens[0] = -5
    out = D.run()
    assert mla.mla_get_device_error()[0] == mla.MLA_ERR_OUT_OF_RANGE
    assert (out[0] == 0).all() and torch.equal(out[1:], good[1:])
    D.lens[0] = 64 * D.table.shape[1] + 1
    out = D.run()
    assert mla.mla_get_device_error()[0] == mla.MLA_ERR_OUT_OF_RANGE
    assert (out[0] == 0).all() and torch.equal(out[1:], good[1:])
    D.lens[0] = 130
    pages = D.codes.shape[0]
    for bad in (-1, pages, 2 ** 31 - 1):
        keep = int(D.table[1, 2])
        D.table[1, 2] = bad
        out = D.run()
        assert mla.mla_get_device_error()[0] == mla.MLA_ERR_OUT_OF_RANGE
        D.table[1, 2] = keep
        # its tokens are zero rows: what a page of zeros gives
        codes = D.codes.clone()
        codes[keep] = 0
        want = plain_decode(D.qn, D.qr, codes, D.scales, D.table, D.lens, D.uk, D.uv)
        assert_close(out.float(), want, "bf16", f"page {bad}")
    assert torch.equal(D.run(), good)
    assert mla.mla_get_device_error() == (0, 0)


def test_equal_calls_give_equal_bits_and_another_stream_works():
    D = Decode(128, 1, [5000, 1, 777] * 5, seed=34)
    want = D.run()
    for _ in range(5):
        assert torch.equal(D.run(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = D.run(ws=D.workspace())
    s.synchronize()
    assert torch.equal(out, want)


def test_two_captured_graphs_replay_on_new_inputs():
    Ds = [Decode(128, 1, [300, 64, 1000], seed=35), Decode(16, 2, [200, 15, 900], seed=36)]
    outs, graphs = [], []
    for D in Ds:
        outs.append(D.run())
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            D.run(out=outs[-1])
        graphs.append(g)
    for step in range(3):
        for D in Ds:
            D.qn.copy_(torch.randn(D.qn.shape, generator=gen(step), device=DEV))
            D.lens.sub_(3)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for D, o in zip(Ds, outs):
            D.check(f"replay {step}", o)


def test_pages_past_four_gigabytes():
    pages = 2 ** 32 // (PAGE * ROW) + 100
    D = Decode(16, 1, [200, 64], seed=37)
    codes = torch.empty(pages, PAGE, ROW, dtype=torch.uint8, device=DEV)
    scales = torch.ones(pages, device=DEV)
    shift = pages - D.codes.shape[0]
    codes[shift:], scales[shift:] = D.codes, D.scales
    want = D.run()
    D.codes, D.scales, D.table = codes, scales, D.table + shift
    assert torch.equal(D.run(), want)
    c = torch.ones(1, DC, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(1, DR, dtype=torch.bfloat16, device=DEV)
    mla.mla_append_paged_q8(D.d, c, k, i32([0, 1]), i32([1]), codes, scales, i32([[pages - 1]]))
    assert float(scales[pages - 1]) == 2.0 ** -8 and (codes[pages - 1, 0, :DC].view(E4M3).float() == 256).all()
    assert mla.mla_get_device_error() == (0, 0)


def test_refused_tensors():
    D = Decode(16, 1, [100], seed=38)
    out = D.run()
    call = lambda **k: mla.mla_decode_absorbed_paged_q8(  # noqa: E731
        **{**dict(dims=D.d, weights=D.w, codes=D.codes, scales=D.scales, block_table=D.table, seq_lens=D.lens, out=out,
                  ws=D.ws, q_nope=D.qn, q_rope=D.qr), **k})
    call()
    for k in (dict(codes=D.codes.view(E4M3)), dict(scales=D.scales[:-1]), dict(scales=D.scales.double()),
              dict(block_table=D.table.long()), dict(seq_lens=D.lens.long()), dict(out=out.float()),
              dict(q_nope=D.qn.float()), dict(q_nope=D.qn[..., :64]), dict(q_rope=D.qr[:, :, :8]),
              dict(q_nope=D.qn.transpose(1, 2)), dict(out=out.cpu()), dict(codes=D.codes[:, ::2])):
        with pytest.raises(ValueError):
            call(**k)
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        call(ws=D.ws[:-256])
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == (0, 0)


@pytest.mark.parametrize("H,Q,B", [(16, 1, 1100), (128, 20, 30), (128, 9, 3), (5, 3, 600)])
def test_more_sequences_or_groups_than_threads(H, Q, B):
    """The work split past one round of the planner, and groups walked one after another."""
    lens = [(37 * i) % 210 for i in range(B)]
    Decode(H, Q, lens, seed=51).check(f"H={H} q_len={Q} B={B}")


def test_sequences_that_share_pages():
    D = Decode(64, 1, [300, 300, 140], seed=52)
    D.table[1, :4] = D.table[0, :4]                      # a common prefix of 256 tokens
    D.table[2, :2] = D.table[0, :2]
    D.table[2, 2] = D.table[2, 1]                        # and the same page twice
    D.check("shared pages")


def test_nan_in_a_later_tokens_row_does_not_reach_an_earlier_token():
    for H, Q in ((16, 3), (128, 2)):
        D = Decode(H, Q, [200, 66], seed=53)
        want = D.run()
        for b, n in enumerate([200, 66]):                # the last new token's row
            D.codes[int(D.table[b, (n - 1) // PAGE]), (n - 1) % PAGE, 3] = 0xFF
        out = D.run()
        assert mla.mla_get_device_error() == (0, 0)
        assert torch.equal(out[:, :-1], want[:, :-1])
        assert torch.isnan(out[:, -1]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_query_value_stays_in_its_row(bad):
    D = Decode(20, 2, [300, 70], seed=54)
    want = D.run()
    D.qn[1, 0, 7, 5] = bad
    D.qr[0, 1, 19, 63] = bad
    out = D.run()
    assert mla.mla_get_device_error() == (0, 0)
    hit = torch.zeros(2, 2, 20, dtype=torch.bool, device=DEV)
    hit[1, 0, 7] = hit[0, 1, 19] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], want[~hit])


@pytest.mark.parametrize("gain", [0.0, 1e-20, 1e-3, 30.0, 1e4])
def test_query_sizes(gain):
    """Rows of very different size in one group: each has its own scale."""
    D = Decode(64, 1, [400, 129], seed=55)
    D.qn[:, :, ::3] *= gain
    D.qr[:, :, ::3] *= gain
    if gain <= 1.0:
        D.check(f"gain {gain}")
        return
    # huge scores: the softmax is nearly one-hot, and an output differs by the error of the
    # scores' difference of its first two keys; only the rows of ordinary size are compared
    got, want = D.run(), D.plain()
    assert mla.mla_get_device_error() == (0, 0) and torch.isfinite(got.float()).all()
    keep = torch.arange(64, device=DEV) % 3 != 0
    assert_close(got[:, :, keep].float(), want[:, :, keep], "bf16", f"gain {gain}, other rows")


def test_two_calls_at_once_with_a_workspace_each():
    Ds = [Decode(128, 1, [3000, 10, 400], seed=56), Decode(16, 4, [900] * 5, seed=57)]
    want = [D.run() for D in Ds]
    streams = [torch.cuda.Stream() for _ in Ds]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for D, s, o in zip(Ds, streams, outs):
            with torch.cuda.stream(s):
                D.run(out=o)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == (0, 0)
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_empty_calls_are_no_ops():
    D = Decode(16, 1, [5], seed=58)
    none = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device=DEV)  # noqa: E731
    mla.mla_decode_absorbed_paged_q8(D.d, D.w, D.codes, D.scales, none(0, 3, t=torch.int32), none(0, t=torch.int32),
                                     none(0, 1, 16, 128), D.ws, none(0, 1, 16, 128), none(0, 1, 16, 64))
    codes, scales = D.codes.clone(), D.scales.clone()
    mla.mla_append_paged_q8(D.d, none(0, DC), none(0, DR), i32([0, 0]), i32([5]), D.codes, D.scales, D.table)
    cache = torch.ones(2, PAGE, ROW, dtype=torch.bfloat16, device=DEV)
    mla.mla_append_paged(D.d, none(0, DC), none(0, DR), i32([0, 0]), i32([5]), cache, D.table)
    assert torch.equal(D.codes, codes) and torch.equal(D.scales, scales) and (cache == 1).all()
    out = Decode(16, 2, [0, 0], seed=59).run()
    assert (out == 0).all() and mla.mla_get_device_error() == (0, 0)


def test_appends_captured_and_replayed():
    """A step's append in a graph, replayed with new rows and lengths in the same buffers."""
    B, steps = 5, 70
    g = gen(60)
    c, k = torch.empty(B, DC, dtype=torch.bfloat16, device=DEV), torch.empty(B, DR, dtype=torch.bfloat16, device=DEV)
    off, lens = i32(list(range(B + 1))), i32([1, 60, 64, 128, 3])
    table, pages = page_table([n + steps for n in lens.tolist()], g)
    codes = torch.zeros(pages, PAGE, ROW, dtype=torch.uint8, device=DEV)
    scales = torch.ones(pages, device=DEV)
    same, same_s = codes.clone(), scales.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mla.mla_append_paged_q8(dims(), c, k, off, lens, codes, scales, table)
    for step in range(steps):
        c.copy_(torch.randn(B, DC, generator=g, device=DEV) * (1 + step % 7))
        k.copy_(torch.randn(B, DR, generator=g, device=DEV))
        graph.replay()
        mla.mla_append_paged_q8(dims(), c, k, off, lens, same, same_s, table)
        lens += 1
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == (0, 0)
    assert torch.equal(codes, same) and torch.equal(scales, same_s)


# ----------------------------------------------------------------- the run of them

def test_prefill_append_steps_and_decode_together():
    """As a server uses them: prompts into fresh 8-bit pages, then steps of one token appended
    and attended to; and the same rows in bf16 pages read by the bf16 paged decode."""
    H, g = 128, gen(41)
    lens = [130, 1, 64, 500]
    B, steps = len(lens), 3
    full = [n + steps for n in lens]
    table, pages = page_table(full, g)
    uk, uv = weights_of(H, 42)
    d = dims(H)
    w = mla.mla_absorb_weights(d, uk, uv)
    codes = torch.full((pages, PAGE, ROW), 0x7F, dtype=torch.uint8, device=DEV)
    scales = torch.full((pages,), float("nan"), device=DEV)
    cache = torch.full((pages, PAGE, ROW), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = mla.workspace(mla.mla_decode_q8_workspace_size(d, B))
    ws16 = mla.workspace(mla.mla_decode_workspace_size(d, B))
    history = [torch.zeros(0, ROW, dtype=torch.float64, device=DEV) for _ in range(B)]
    now = [0] * B
    for step in range(steps + 1):
        new = lens if step == 0 else [1] * B
        n = sum(new)
        kv = (torch.randn(n, ROW, generator=g, device=DEV) * (0.3 + 0.4 * step)).to(torch.bfloat16)
        off, after = i32([0] + list(np.cumsum(new))), [a + k for a, k in zip(now, new)]
        args = (d, kv[:, :DC], kv[:, DC:], off, i32(after))
        mla.mla_append_paged_q8(*args, codes, scales, table)
        mla.mla_append_paged(*args, cache, table)
        at = 0
        for b in range(B):
            x = kv[at:at + new[b]]
            r = torch.cat((x[:, :DC].double(), rotate64(x[:, DC:], torch.arange(now[b], after[b], device=DEV))), 1)
            history[b] = torch.cat((history[b], r))
            at += new[b]
        now = after
        qn = torch.randn(B, 1, H, 128, generator=g, device=DEV).to(torch.bfloat16)
        qr = torch.randn(B, 1, H, 64, generator=g, device=DEV).to(torch.bfloat16)
        out = torch.empty(B, 1, H, 128, dtype=torch.bfloat16, device=DEV)
        mla.mla_decode_absorbed_paged_q8(d, w, codes, scales, table, i32(now), out, ws, qn, qr)
        out16 = torch.empty(B, H, 128, dtype=torch.bfloat16, device=DEV)
        mla.mla_decode_absorbed_paged(d, w, cache, table, i32(now), out16, ws16, q_nope=qn[:, 0].contiguous(),
                                      q_rope=qr[:, 0].contiguous())
        assert mla.mla_get_device_error() == (0, 0)
        assert_close(out.float(), plain_decode(qn, qr, codes, scales, table, now, uk, uv), "bf16", f"8-bit step {step}")
        for b in range(B):
            # The bf16 decode adds two half scores (columns split in two), each rounded to bf16:
            # a score is off by up to e = 2^-8 (|half| + |half|) SCALE.  With weights
            # p_j e^(d_j) / sum p e^d, |d_j| <= e, every weight is off by a factor within
            # e^(+-2e), so an output by up to (e^(2e) - 1) sum_j p_j |v_j|, beside the bf16 tolerance.
            ql = torch.einsum("hj,hjc->hc", qn[b, 0].double(), uk.double())
            q, rows = torch.cat((ql, qr[b, 0].double()), -1), history[b]
            halves = [q[:, i] @ rows[:, i].T for i in (list(range(256)) + list(range(512, 544)),
                                                       list(range(256, 512)) + list(range(544, 576)))]
            p = torch.softmax(SCALE * (halves[0] + halves[1]), -1)
            want = torch.einsum("hc,hvc->hv", p @ rows[:, :DC], uv.double())
            e = 2.0 ** -8 * SCALE * (halves[0].abs() + halves[1].abs()).amax(-1)
            v = torch.einsum("nc,hvc->hnv", rows[:, :DC], uv.double())
            lim = 2e-2 * want.pow(2).mean(-1, keepdim=True).sqrt() + \
                (torch.exp(2 * e) - 1)[:, None] * torch.einsum("hn,hnv->hv", p, v.abs())
            assert ((out16[b].double() - want).abs() <= lim).all(), f"bf16 step {step} sequence {b}"
            # codes hold the rows to E4M3 precision
            pg = table[b, :(now[b] + 63) // 64].long()
            held = (code_values(codes[pg]) * scales[pg].double()[:, None, None]).reshape(-1, ROW)[:now[b]]
            top = scales[pg].double().repeat_interleave(PAGE)[:now[b], None]
            assert ((held - history[b]).abs() <= 2.0 ** -4 * 1.01 * history[b].abs() + 2.0 ** -8 * top).all()
