"""Refusals of the paged entry points, on the host (no GPU is touched: fake,
never-dereferenced addresses, or CPU tensors)."""
import pytest
import torch

import full_gqa_learned_b200 as fa
from full_gqa_learned_b200 import build

A = 0x100000
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fa.load_library()


BASE = dict(k=A, v=A, wk=A, kp=A, vp=A, ks=None, vs=None, table=A, len=A, cu=A, B=2, T=8, max_pages=4, pages=9, ps=16, g=4,
            rope=1, theta=1e4, eps=1e-6, ws=A, ws_bytes=1 << 40, q=A, wq=A, sinks=A, max_new=4, window=513, out=A, lse=A)


def append(lib, **kw):
    a = dict(BASE, **kw)
    return lib.flint_paged_append(a["k"], a["v"], a["wk"], a["kp"], a["vp"], a["ks"], a["vs"], a["table"], a["len"], a["cu"],
                                  a["B"], a["T"], a["max_pages"], a["pages"], a["ps"], a["g"], a["rope"], a["theta"], a["eps"],
                                  a["ws"], a["ws_bytes"], None)


def read(lib, **kw):
    a = dict(BASE, **kw)
    return lib.flint_paged_read(a["kp"], a["vp"], a["ks"], a["vs"], a["table"], a["len"], a["cu"], a["B"], a["T"],
                                a["max_pages"], a["pages"], a["ps"], a["g"], a["k"], a["v"], a["ws"], a["ws_bytes"], None)


def attn(lib, **kw):
    a = dict(BASE, **kw)
    return lib.flint_attn_paged(a["q"], a["wq"], a["sinks"], a["kp"], a["vp"], a["ks"], a["vs"], a["table"], a["len"], a["cu"],
                                a["B"], a["T"], a["max_new"], a["max_pages"], a["pages"], a["ps"], a["g"], a["window"],
                                a["rope"], a["theta"], a["eps"], a["out"], a["lse"], a["ws"], a["ws_bytes"], None)


SHARED = [(dict(B=-1), INVALID), (dict(B=1 << 16), INVALID), (dict(T=-1), INVALID), (dict(T=(1 << 24) + 1), INVALID),
          (dict(g=3), INVALID), (dict(g=0), INVALID), (dict(ps=8), UNSUPPORTED), (dict(ps=48), UNSUPPORTED),
          (dict(ps=256), UNSUPPORTED), (dict(max_pages=0), INVALID), (dict(pages=0), INVALID), (dict(pages=1 << 30), INVALID),
          (dict(ks=A), INVALID), (dict(vs=A), INVALID), (dict(kp=None), INVALID), (dict(vp=None), INVALID),
          (dict(table=None), INVALID), (dict(len=None), INVALID), (dict(cu=None), INVALID), (dict(kp=A + 8), INVALID),
          (dict(vp=A + 2), INVALID), (dict(ks=A + 1, vs=A), INVALID), (dict(table=A + 2), INVALID), (dict(cu=A + 1), INVALID),
          (dict(ws=None), WORKSPACE), (dict(ws=A + 16), WORKSPACE), (dict(ws_bytes=8), WORKSPACE)]
ROPE = [(dict(rope=2), INVALID), (dict(theta=1.0), INVALID), (dict(theta=float("inf")), INVALID), (dict(eps=0.0), INVALID),
        (dict(eps=float("nan")), INVALID)]


@pytest.mark.parametrize("kw,want", SHARED + ROPE + [(dict(k=None), INVALID), (dict(v=A + 8), INVALID), (dict(wk=None), INVALID),
                                                     (dict(wk=A + 2), INVALID)])
def test_append_refuses(lib, kw, want):
    assert append(lib, **kw) == want
    assert lib.flint_attn_last_error() != b""


@pytest.mark.parametrize("kw,want", SHARED + [(dict(k=None), INVALID), (dict(v=A + 8), INVALID)])
def test_read_refuses(lib, kw, want):
    assert read(lib, **kw) == want


@pytest.mark.parametrize("kw,want", SHARED + ROPE + [(dict(q=None), INVALID), (dict(q=A + 8), INVALID), (dict(wq=None), INVALID),
                                                     (dict(sinks=None), INVALID), (dict(out=None), INVALID),
                                                     (dict(out=A + 4), INVALID), (dict(lse=A + 1), INVALID),
                                                     (dict(window=-1), INVALID), (dict(max_new=-1), INVALID)])
def test_attn_refuses(lib, kw, want):
    assert attn(lib, **kw) == want


@pytest.mark.parametrize("call", [append, read, attn])
@pytest.mark.parametrize("kw", [dict(B=0), dict(T=0), dict(B=0, kp=None, ws=None)])
def test_nothing_to_do(lib, call, kw):
    assert call(lib, **kw) == 0


def test_workspace_sizes(lib):
    ws = fa.paged_workspace_bytes
    assert 0 < ws(128, 128, 1, 4096, 64) < 8 << 20                       # a decode step: partials of the CTAs
    least = ws(4, 2048, 512, 100, 64, window=0)
    full = ws(4, 2048, 512, 100, 64, window=0, eight_bit=True)
    assert full == least + 4 * 6400 * 4 * 512                            # room for every position in 16 bits
    assert ws(4, 2048, 512, 100000, 64, window=0, eight_bit=True) == ws(4, 2048, 512, 100000, 64, window=0)   # over 512 MiB
    assert ws(4, 2048, 512, 100000, 64, window=513, eight_bit=True) < least + (64 << 20)
    assert ws(4, 8, 4, 100, 64, eight_bit=True) == ws(4, 8, 4, 100, 64)
    for bad in ((-1, 1, 1, 1, 16), (1, -1, 1, 1, 16), (1, 1, -1, 1, 16), (1, 1, 1, 0, 16), (1, 1, 1, 1, 24)):
        assert ws(*bad) == 0
    assert ws(1, 1, 1, 1, 16, kv_heads=3) == 0 and ws(1, 1, 1, 1, 16, window=-1) == 0


def test_workspace_is_checked_against_the_call(lib):
    need = fa.paged_workspace_bytes(2, 8, 4, 4, 16)
    assert attn(lib, ws_bytes=need - 1) == WORKSPACE
    need = fa.paged_workspace_bytes(2, 64, 32, 4, 16)
    assert attn(lib, T=64, max_new=32, ws_bytes=need - 1) == WORKSPACE
    assert append(lib, ws_bytes=255) == WORKSPACE


def cpu_args():
    t = dict(k=torch.zeros(3, 4, 128, dtype=torch.bfloat16), v=torch.zeros(3, 4, 128, dtype=torch.bfloat16), w=torch.ones(128),
             kp=torch.zeros(5, 4, 16, 128, dtype=torch.float16), vp=torch.zeros(5, 4, 16, 128, dtype=torch.bfloat16),
             table=torch.zeros(2, 3, dtype=torch.int32), len=torch.zeros(2, dtype=torch.int32), cu=torch.zeros(3, dtype=torch.int32))
    return t


def test_binding_refuses_cpu_tensors_and_mixed_formats(lib):
    t = cpu_args()
    with pytest.raises(ValueError, match="CUDA"):
        fa.paged_append(t["k"], t["v"], t["w"], t["kp"], t["vp"], t["table"], t["len"], t["cu"])
    with pytest.raises(ValueError, match="neither"):
        fa.paged_append(t["k"], t["v"], t["w"], t["kp"], t["vp"], t["table"], t["len"], t["cu"],
                        k_scales=torch.zeros(5, 4, 16, dtype=torch.float8_e8m0fnu))
    with pytest.raises(ValueError, match="k_pages"):
        fa.paged_read(t["kp"][0], t["vp"], t["table"], t["len"], t["cu"], 3)
    with pytest.raises(ValueError, match="k_pages"):
        fa.paged_read(t["kp"][..., :64], t["vp"], t["table"], t["len"], t["cu"], 3)
