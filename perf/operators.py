"""Cases of the paged-cache operators: appending given latents to a paged cache (bf16 rows, and
8-bit codes with one scale per 64-token page) and absorbed attention over the 8-bit cache.

`run` computes a case in its plain form (elementary torch operations in 32 bits), or through
the library where `own` is true.  `exact` restates the definitions in 64 bits.

The cache: pages of 64 tokens; sequence b's tokens 64 j .. 64 j + 63 are page block_table[b, j].
A row is [c (512) | rotated key (64)].  The 8-bit cache holds a row as 576 FP8 E4M3 codes, and
one fp32 scale per page (one latent head is shared by all query heads), a power of two:
value = code * scale.
"""
import math
import random

import torch

own = False

PAGE, DC, DR, ROW, NOPE, VH = 64, 512, 64, 576, 128, 128
SCALE = 1.0 / math.sqrt(NOPE + DR)
THETA = 10000.0


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 64 sequences: one new token each, at ragged positions (latency)
        _append("append_step_b64", "append", 64, 1, 1, 0, 4096, 11),
        # a prefill of the V2 prompt shape: four prompts of 4096 tokens into empty pages
        _append("append_prefill_b4_s4096", "append", 4, 4096, 4096, 0, 0, 12),
        # the same step into the 8-bit cache: every token joins a page that others hold a part of
        _append("append_q8_step_b64", "append_q8", 64, 1, 1, 0, 4096, 13),
        # ragged chunks behind ragged prefixes (chunked prefill), page borders inside the chunks
        _append("append_q8_chunks_b7", "append_q8", 7, 1, 1000, 0, 2000, 14),
        # the prefill into the 8-bit cache
        _append("append_q8_prefill_b4_s4096", "append_q8", 4, 4096, 4096, 0, 0, 15),
        # one user, a short context: what a step costs before the cache matters
        _decode("decode_q8_b1_ctx100", 1, 1, 128, 100, 100, 21),
        # one user, a long context: one sequence over the whole GPU
        _decode("decode_q8_b1_ctx32768", 1, 1, 128, 32768, 32768, 22),
        # the V3 decode shape: 32 sequences of 4096 tokens, 128 heads
        _decode("decode_q8_b32_ctx4096", 32, 1, 128, 4096, 4096, 23),
        # one GPU's 16 heads of a head-parallel layer, ragged odd lengths from empty up
        _decode("decode_q8_h16_b48_ragged", 48, 1, 16, 0, 9001, 24),
        # verification of draft tokens: two new tokens per sequence
        _decode("decode_q8_q2_b32_ctx4096", 32, 2, 128, 4096, 4096, 25),
        # a chunk of 100 new tokens behind a cached prefix, 64 heads per GPU
        _decode("decode_q8_h64_q100_b2", 2, 100, 64, 3000, 4300, 26),
        # ragged long contexts, as a server with mixed users meets them
        _decode("decode_q8_ragged_b64", 64, 1, 128, 1024, 32768, 27),
    ]


def _append(name, op, B, new_lo, new_hi, pre_lo, pre_hi, lens_seed):
    return {"name": name, "op": op, "B": B, "new_lo": new_lo, "new_hi": new_hi, "pre_lo": pre_lo,
            "pre_hi": pre_hi, "lens_seed": lens_seed}


def _decode(name, B, q_len, H, lo, hi, lens_seed):
    return {"name": name, "op": "decode_q8", "B": B, "q_len": q_len, "H": H, "lo": lo, "hi": hi,
            "lens_seed": lens_seed}


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append_q8", "decode_q8", "decode_q8"])
    seed = rng.randrange(1 << 30)
    if op != "decode_q8":
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, min(4096, 16384 // B))
        lo = rng.choice([hi, rng.randint(1, hi)])
        pre = rng.choice([0, rng.randint(1, 4096)])
        c = _append("", op, B, lo, hi, rng.randint(0, pre), pre, seed)
    else:
        H = rng.choice([128, 128, 64, 32, 16, rng.randint(1, 128)])
        B = _log_int(rng, 1, 64)
        q_len = rng.choice([1, 1, 1, 2, rng.randint(3, 8), _log_int(rng, 9, 128)])
        q_len = max(1, min(q_len, 256 // B))
        # at most the tokens and products of the ragged listed case
        hi = _log_int(rng, 1, max(64, min(32768, 64 * 16384 * 128 // (B * q_len * H), (1 << 20) // B)))
        lo = rng.choice([hi, rng.randint(0, hi)])
        c = _decode("", B, q_len, H, lo, hi, seed)
    del c["name"]
    return c


def _lens(case):
    """Per sequence: (tokens before, new tokens) of an append, or cached tokens of a decode."""
    r = random.Random(case["lens_seed"])
    if case["op"] == "decode_q8":
        return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    return [(r.randint(case["pre_lo"], case["pre_hi"]), r.randint(case["new_lo"], case["new_hi"]))
            for _ in range(case["B"])]


def work(case):
    lens = _lens(case)
    if case["op"] == "decode_q8":
        B, Q, H = case["B"], case["q_len"], case["H"]
        tokens = sum(lens)
        keys = sum(max(0, n - (Q - 1 - t)) for n in lens for t in range(Q))   # (query token, key) pairs
        pages = sum((n + PAGE - 1) // PAGE for n in lens)
        rows = B * Q * H
        byts = tokens * ROW + pages * 8 + B * 4 + rows * (NOPE + DR + VH) * 2 + H * (NOPE + VH) * DC * 2
        return {"bytes": byts, "flops": 2 * H * keys * (ROW + DC) + 2 * rows * DC * (NOPE + VH)}
    n = sum(k for _, k in lens)
    pages = sum((a + k + PAGE - 1) // PAGE - a // PAGE for a, k in lens)
    elem = 2 if case["op"] == "append" else 1
    byts = n * ROW * (2 + elem) + len(lens) * 8 + pages * (4 if elem == 2 else 12)
    return {"bytes": byts, "flops": n * DR * 3}


# --------------------------------------------------------------------------- inputs

def _block_table(lens, gen, dev):
    """Pages in random order, with a few spare ones, and the table of them."""
    blocks = [(n + PAGE - 1) // PAGE for n in lens]
    total = sum(blocks)
    num_pages = total + 8
    perm = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)
    first = torch.tensor([0] + blocks, device=dev).cumsum(0)[:-1]
    width = max(max(blocks), 1)
    col = torch.arange(width, device=dev)
    at = (first[:, None] + col[None, :]).clamp_(max=num_pages - 1)
    table = torch.where(col[None, :] < torch.tensor(blocks, device=dev)[:, None], perm[at], 0)
    return table.to(torch.int32).contiguous(), num_pages


def _pow2_scale(amax):
    """Smallest power of two s with amax <= 448 s (1 for 0), at least 2^-60."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), torch.where(m <= 0.875, e - 9, e - 8))
    return torch.where(amax > 0, s.clamp(min=2.0 ** -60), torch.ones_like(s))


def _page_values(k, gen, dev):
    """k pages of cache values: tokens of slightly different size, larger rotary parts."""
    x = torch.randn(k, PAGE, ROW, generator=gen, device=dev) * 0.5
    x *= torch.exp(0.3 * torch.randn(k, PAGE, 1, generator=gen, device=dev))
    x[..., DC:] *= 2.0
    return x


def _pages_q8(num_pages, gen, dev):
    """A cache of the 8-bit form, every page full (what lies past a sequence's end is stale)."""
    codes = torch.empty(num_pages, PAGE, ROW, dtype=torch.uint8, device=dev)
    scales = torch.empty(num_pages, device=dev)
    for a in range(0, num_pages, 4096):
        x = _page_values(min(4096, num_pages - a), gen, dev)
        s = _pow2_scale(x.abs().amax((1, 2)))
        codes[a:a + len(x)] = (x / s[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[a:a + len(x)] = s
    return codes, scales


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": case}
    lens = _lens(case)
    if case["op"] == "decode_q8":
        B, Q, H = case["B"], case["q_len"], case["H"]
        s["table"], num_pages = _block_table(lens, gen, dev)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["codes"], s["scales"] = _pages_q8(num_pages, gen, dev)
        rnd = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731
        s["q_nope"] = rnd(B, Q, H, NOPE).to(torch.bfloat16)
        s["q_rope"] = rnd(B, Q, H, DR).to(torch.bfloat16)
        s["W_UK"] = (rnd(H, NOPE, DC) / math.sqrt(DC)).to(torch.bfloat16)
        s["W_UV"] = (rnd(H, VH, DC) / math.sqrt(DC)).to(torch.bfloat16)
        if own:
            import compressed_kv_cache_absorbed_b200 as mla
            s["dims"] = mla.make_dims(H, 0, DC, DR, NOPE, VH, torch.bfloat16)
            s["weights"] = mla.mla_absorb_weights(s["dims"], s["W_UK"], s["W_UV"])
            s["ws"] = mla.workspace(mla.mla_decode_q8_workspace_size(s["dims"], B, Q), dev)
            s["out"] = torch.empty(B, Q, H, VH, dtype=torch.bfloat16, device=dev)
        return s
    total = [a + k for a, k in lens]
    s["table"], num_pages = _block_table(total, gen, dev)
    s["lens"] = torch.tensor(total, dtype=torch.int32, device=dev)      # after the append
    s["new"] = torch.tensor([0] + [k for _, k in lens], device=dev).cumsum(0).to(torch.int32)
    # the down-projection's output [n, 576]: the latent and the unrotated key are slices of it
    n = sum(k for _, k in lens)
    kv = _page_values((n + PAGE - 1) // PAGE, gen, dev).reshape(-1, ROW)[:n].to(torch.bfloat16)
    s["c"], s["k_r"] = kv[:, :DC], kv[:, DC:]
    if case["op"] == "append":
        s["cache"] = _page_values(num_pages, gen, dev).to(torch.bfloat16)
    else:
        s["codes"], s["scales"] = _pages_q8(num_pages, gen, dev)
    if own:
        import compressed_kv_cache_absorbed_b200 as mla
        s["dims"] = mla.make_dims(128, 0, DC, DR, NOPE, VH, torch.bfloat16)
    return s


# ----------------------------------------------------------------------- plain forms

def _rotated(k_r, pos):
    """Pairs (2i, 2i+1) rotated by pos * theta^(-2i/64): angles and products in 64 bits."""
    freq = THETA ** (-torch.arange(0, DR, 2, device=pos.device, dtype=torch.float64) / DR)
    ang = pos.double()[:, None] * freq[None, :]
    co, si = ang.cos(), ang.sin()
    x = k_r.double()
    a, b = x[:, 0::2], x[:, 1::2]
    return torch.stack((a * co - b * si, a * si + b * co), -1).flatten(1).float()


def _places(s):
    """Of every new token: its position in its sequence, its page and its row in the page."""
    new, lens, table = s["new"].long(), s["lens"].long(), s["table"].long()
    i = torch.arange(s["c"].shape[0], device=new.device)
    b = torch.searchsorted(new, i, right=True) - 1
    pos = lens[b] - (new[b + 1] - i)
    return pos, table[b, pos // PAGE], pos % PAGE


def _plain_append(s):
    pos, page, row = _places(s)
    s["cache"][page, row] = torch.cat((s["c"].float(), _rotated(s["k_r"], pos)), 1).to(torch.bfloat16)
    return s["cache"]


def _plain_append_q8(s):
    pos, page, row = _places(s)
    codes, scales = s["codes"], s["scales"]
    x = torch.cat((s["c"].float(), _rotated(s["k_r"], pos)), 1)
    # the scale each touched page needs for its new tokens
    amax = torch.zeros_like(scales).scatter_reduce_(0, page, x.abs().amax(1), "amax")
    need = _pow2_scale(amax)
    # pages that hold earlier tokens keep at least their scale; if it grows, those are rescaled
    new, lens = s["new"].long(), s["lens"].long()
    start = lens - (new[1:] - new[:-1])
    held = start % PAGE
    at = s["table"].long().gather(1, (start // PAGE).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0]
    joins = held > 0
    grown = torch.where(joins, torch.maximum(need[at], scales[at]), need[at])
    old = codes[at]
    again = (old.view(torch.float8_e4m3fn).float() * (scales[at] / grown)[:, None, None]).to(torch.float8_e4m3fn)
    rows = torch.arange(PAGE, device=codes.device)[None, :, None]
    # a sequence that joins no page writes its first page's rows back as they were
    codes[at] = torch.where(joins[:, None, None] & (rows < held[:, None, None]), again.view(torch.uint8), old)
    scales[page] = need[page]
    scales[at] = torch.where(new[1:] > new[:-1], grown, scales[at])
    codes[page, row] = (x / scales[page][:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scales


def _plain_decode_q8(s):
    B, Q, H, _ = s["q_nope"].shape
    q_lat = torch.einsum("bqhj,hjc->bqhc", s["q_nope"].float(), s["W_UK"].float())
    q = torch.cat((q_lat, s["q_rope"].float()), -1).reshape(B, Q * H, ROW)
    table = s["table"].long()
    kv = s["codes"][table].view(torch.float8_e4m3fn).float() * s["scales"][table][:, :, None, None]
    kv = kv.reshape(B, -1, ROW)
    p = torch.bmm(q, kv.transpose(1, 2)).mul_(SCALE).view(B, Q, H, -1)
    limit = s["lens"].long()[:, None] - (Q - 1) + torch.arange(Q, device=q.device)[None, :]
    gone = torch.arange(kv.shape[1], device=q.device)[None, None, :] >= limit[:, :, None]
    p.masked_fill_(gone[:, :, None, :], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total > 0, total, 1.0))
    o_lat = torch.bmm(p.view(B, Q * H, -1), kv[..., :DC]).view(B, Q, H, DC)
    return torch.einsum("bqhc,hvc->bqhv", o_lat, s["W_UV"].float()).to(torch.bfloat16)


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import compressed_kv_cache_absorbed_b200 as mla
        if op == "append":
            mla.mla_append_paged(s["dims"], s["c"], s["k_r"], s["new"], s["lens"], s["cache"], s["table"])
            return s["cache"]
        if op == "append_q8":
            mla.mla_append_paged_q8(s["dims"], s["c"], s["k_r"], s["new"], s["lens"], s["codes"], s["scales"],
                                    s["table"])
            return s["codes"].view(torch.float8_e4m3fn), s["scales"]
        mla.mla_decode_absorbed_paged_q8(s["dims"], s["weights"], s["codes"], s["scales"], s["table"], s["lens"],
                                         s["out"], s["ws"], s["q_nope"], s["q_rope"])
        return s["out"]
    if op == "append":
        return _plain_append(s)
    if op == "append_q8":
        codes, scales = _plain_append_q8(s)
        return codes.view(torch.float8_e4m3fn), scales
    return _plain_decode_q8(s)


# --------------------------------------------------------------- definitions in 64 bits

def _e4m3_values(codes):
    """The numbers that E4M3 bytes stand for: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    k = codes.to(torch.int32)
    e, m = (k >> 3) & 15, (k & 7).double()
    mag = torch.where(e > 0, torch.ldexp(1 + m / 8, e - 7), m * 2.0 ** -9)
    return torch.where(k >= 128, -mag, mag)


def exact(case, seed):
    s = prepare(case, seed)
    table, lens = s["table"].tolist(), s["lens"].tolist()
    if case["op"] == "decode_q8":
        Q = case["q_len"]
        out = torch.zeros(case["B"], Q, case["H"], VH, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            if n == 0:
                continue
            pages = torch.tensor(table[b][:(n + PAGE - 1) // PAGE], device="cuda")
            rows = (_e4m3_values(s["codes"][pages]) * s["scales"][pages].double()[:, None, None]).reshape(-1, ROW)[:n]
            q_lat = torch.einsum("qhj,hjc->hqc", s["q_nope"][b].double(), s["W_UK"].double())
            # heads in groups, so that the scores of a long chunk fit
            for h0 in range(0, case["H"], 16):
                hs = slice(h0, h0 + 16)
                z = q_lat[hs] @ rows[:, :DC].T + s["q_rope"][b].double().transpose(0, 1)[hs] @ rows[:, DC:].T
                z = z / math.sqrt(192.0)
                seen = torch.arange(n, device="cuda")[None, :] < (n - Q + 1 + torch.arange(Q, device="cuda"))[:, None]
                z = torch.where(seen[None], z, -math.inf)
                w = torch.where(seen.any(1)[None, :, None], torch.softmax(z, -1), 0.0)
                v = torch.einsum("hqc,hvc->qhv", w @ rows[:, :DC], s["W_UV"][hs].double())
                out[b, :, hs] = v
        return out
    new = s["new"].tolist()
    i = torch.arange(0, DR, 2, dtype=torch.float64, device="cuda")
    q8 = case["op"] == "append_q8"
    if q8:
        codes, scales = _e4m3_values(s["codes"]), s["scales"].double()
    else:
        cache = s["cache"].double()
    for b, n in enumerate(lens):
        k = new[b + 1] - new[b]
        pos = torch.arange(n - k, n, device="cuda")
        c = s["c"][new[b]:new[b + 1]].double()
        z = torch.view_as_complex(s["k_r"][new[b]:new[b + 1]].double().reshape(k, DR // 2, 2).contiguous())
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda").expand(k, DR // 2),
                           pos[:, None] * torch.exp(-i / DR * math.log(THETA)))
        row = torch.cat((c, torch.view_as_real(z * turn).reshape(k, DR)), 1)
        for j in range((n - k) // PAGE, (n - 1) // PAGE + 1):
            a, e = max(n - k, j * PAGE), min(n, (j + 1) * PAGE)
            x, page = row[a - (n - k):e - (n - k)], table[b][j]
            if not q8:
                cache[page, a - j * PAGE:e - j * PAGE] = x
                continue
            top = float(x.abs().max())
            scale = 1.0 if top == 0 else max(2.0 ** -60, 2.0 ** math.ceil(math.log2(top / 448)))
            if a > j * PAGE:   # earlier tokens are here
                before = float(scales[page])
                scale = max(scale, before)
                codes[page, :a - j * PAGE] *= before / scale
            scales[page] = scale
            codes[page, a - j * PAGE:e - j * PAGE] = x / scale   # what the 8-bit codes round
    return (codes, scales) if q8 else cache
