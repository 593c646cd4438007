"""The paged append's split into page items (csrc/paged_plan.h), compiled for the host and
compared with a plain walk over the tokens; and the refusals of the paged-cache calls (no GPU
needed: nothing here launches a kernel)."""
from __future__ import annotations

import ctypes
import os
import random
import subprocess

import pytest
import torch

import compressed_kv_cache_absorbed_b200 as mla

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHIM = """
#include "paged_plan.h"
extern "C" int item(int o0, int o1, int len, int mb, long long k, int* out) {
    mla::AppendItem it{};
    const int r = mla::append_item(o0, o1, len, mb, k, &it);
    out[0] = it.block; out[1] = it.r0; out[2] = it.r1; out[3] = it.src;
    return r;
}
extern "C" long long base(int o0, int b) { return mla::append_item_base(o0, b); }
extern "C" long long items(int n, int B) { return mla::append_items(n, B); }
extern "C" int offsets_ok(int o0, int o1, int b, int B, int n) { return mla::append_offsets_ok(o0, o1, b, B, n); }
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "compressed_kv_cache_absorbed_b200", "csrc"), str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    for f in (lib.base, lib.items):
        f.restype = ctypes.c_longlong
    lib.item.argtypes = [ctypes.c_int] * 4 + [ctypes.c_longlong, ctypes.POINTER(ctypes.c_int)]
    return lib


def walk(plan, new, lens, mb):
    """(sequence, token, input row) triples the items cover, each page at most once."""
    off = [0]
    for k in new:
        off.append(off[-1] + k)
    n, B = off[-1], len(new)
    got, pages, out = [], set(), (ctypes.c_int * 4)()
    for b in range(B):
        first, last = plan.base(off[b], b), plan.base(off[b + 1], b + 1)
        for k in range(last - first):
            if plan.item(off[b], off[b + 1], lens[b], mb, k, out) != 1:
                continue
            block, r0, r1, src = out
            assert 0 <= r0 < r1 <= 64 and (b, block) not in pages
            pages.add((b, block))
            got += [(b, 64 * block + r, src + r - r0) for r in range(r0, r1)]
    assert plan.base(off[0], 0) == 0 and plan.base(n, B) == plan.items(n, B)
    return off, got


@pytest.mark.parametrize("seed", range(40))
def test_items_cover_every_new_token_once(plan, seed):
    r = random.Random(seed)
    B = r.randint(1, 9)
    new = [r.choice([0, 1, r.randint(0, 64), r.randint(0, 400)]) for _ in range(B)]
    pre = [r.choice([0, 1, 63, 64, r.randint(0, 300)]) for _ in range(B)]
    lens = [a + k for a, k in zip(pre, new)]
    off, got = walk(plan, new, lens, mb=20)
    want = [(b, pre[b] + i, off[b] + i) for b in range(B) for i in range(new[b])]
    assert sorted(got) == sorted(want)


def test_invalid_sequences_are_reported_once(plan):
    out = (ctypes.c_int * 4)()
    for o0, o1, ln, mb in ((0, 5, 4, 1), (0, 5, 65, 1), (3, 200, 199 + 64, 4)):
        k = range(plan.base(o1, 1) - plan.base(o0, 0))
        r = [plan.item(o0, o1, ln, mb, i, out) for i in k]
        bad = ln < o1 - o0 or ln > 64 * mb
        assert (r[0] == -1 and all(x == 0 for x in r[1:])) if bad else -1 not in r
    assert plan.offsets_ok(0, 4, 0, 1, 4)
    for o0, o1, b, B, n in ((1, 4, 0, 1, 4), (0, 3, 0, 1, 4), (0, 5, 0, 2, 4), (3, 2, 1, 3, 4), (-1, 2, 1, 3, 4)):
        assert not plan.offsets_ok(o0, o1, b, B, n)


# ------------------------------------------------------------------------ refusals

def dims(H=128, dtype="bf16", **kw):
    d = dict(H=H, d_model=0, d_c=512, d_hR=64, qk_nope=128, v_head=128, dtype=dtype)
    d.update(kw)
    return mla.make_dims(**d)


def test_workspace_size_of_the_8_bit_decode():
    f = mla.mla_decode_q8_workspace_size
    assert 0 < f(dims(16), 1) < f(dims(128), 1) < f(dims(128), 64) < f(dims(128), 64, 4)
    assert f(dims(), 4, 0) == f(dims(), -1, 1) == f(dims(), 65535, 2) == 0
    assert f(dims(H=129), 4) == f(dims(dtype="f32"), 4) == f(dims(d_c=256), 4) == f(dims(v_head=64), 4) == 0


def test_paged_append_argument_errors():
    lib, p = mla.lib(), ctypes.c_void_p(4096)
    I, U, OK = mla.MLA_ERR_INVALID_ARG, mla.MLA_ERR_UNSUPPORTED, mla.MLA_OK

    def bf16(d, c=p, ld_c=576, k=p, ld_k=576, no=p, sl=p, B=2, n=3, cache=p, pages=4, bt=p, mb=2):
        return lib.mla_append_paged(ctypes.byref(d), c, ld_c, k, ld_k, no, sl, None, B, n, cache, pages, bt, mb, None)

    def q8(d, c=p, ld_c=576, k=p, ld_k=576, no=p, sl=p, B=2, n=3, codes=p, sc=p, pages=4, bt=p, mb=2):
        return lib.mla_append_paged_q8(ctypes.byref(d), c, ld_c, k, ld_k, no, sl, None, B, n, codes, sc, pages, bt, mb,
                                       None)

    for call, cache in ((bf16, "cache"), (q8, "codes")):
        assert call(dims(), n=0) == OK
        assert call(dims(), n=-1) == call(dims(), B=-1) == call(dims(), B=0) == I
        for k in ("c", "k", "no", "sl", "bt", cache):
            assert call(dims(), **{k: None}) == I, k
        assert call(dims(), ld_c=511) == call(dims(), ld_k=63) == call(dims(), pages=0) == call(dims(), mb=0) == I
        assert call(dims(), c=ctypes.c_void_p(4097)) == call(dims(), bt=ctypes.c_void_p(4098)) == I
        assert call(dims(), n=2 ** 31 - 1, B=2 ** 31 - 1) == U
        assert call(dims(d_hR=63)) == U
    assert q8(dims(), sc=None) == q8(dims(), codes=ctypes.c_void_p(4104)) == I
    assert q8(dims(dtype="f32")) == q8(dims(d_c=256)) == q8(dims(d_hR=32)) == U


def test_8_bit_decode_argument_errors():
    lib, p = mla.lib(), ctypes.c_void_p(4096)

    def call(d, w=None, B=2, q_len=1):
        return lib.mla_decode_absorbed_paged_q8(ctypes.byref(d), w, p, p, p, p, 4, p, 2, p, B, q_len, p, p, 1 << 30,
                                                None)
    assert call(dims()) == mla.MLA_ERR_INVALID_ARG          # no weights handle
    assert call(dims(d_hR=63)) == mla.MLA_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", ["append", "append_q8", "decode"])
def test_tensors_on_the_host_are_refused(call):
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    i32 = torch.int32
    with pytest.raises(ValueError):
        if call == "append":
            mla.mla_append_paged(dims(), z(1, 512), z(1, 64), z(2, t=i32), z(1, t=i32), z(1, 64, 576), z(1, 1, t=i32))
        elif call == "append_q8":
            mla.mla_append_paged_q8(dims(), z(1, 512), z(1, 64), z(2, t=i32), z(1, t=i32), z(1, 64, 576, t=torch.uint8),
                                    z(1, t=torch.float32), z(1, 1, t=i32))
        else:
            mla.mla_decode_absorbed_paged_q8(dims(), None, z(1, 64, 576, t=torch.uint8), z(1, t=torch.float32),
                                             z(1, 1, t=i32), z(1, t=i32), z(1, 1, 128, 128), z(256, t=torch.uint8),
                                             z(1, 1, 128, 128), z(1, 1, 128, 64))
