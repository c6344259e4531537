"""Host-side argument checks of the rotary paged appends and of the attention
over e4m3 pages (CPU only: every call fails validation, before any CUDA call)."""
import os

import pytest

FAKE = 0x10000          # aligned, never dereferenced
MISALIGNED = 0x10008


@pytest.fixture(scope="module")
def lib():
    from sliding_window_gqa_ring_gb300 import build, carat
    if not os.path.exists(carat.LIBRARY):
        build.build()
    return carat.library()


OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def _rope(lib, fp8, **kw):
    a = dict(kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, num=8, table=FAKE, mp=4, rows=128, R=16, kn=FAKE,
             vn=FAKE, kvs=512, qo=FAKE, q=FAKE, qs=4096, cs=FAKE, trows=512, r=256, il=0, pos=None,
             cnt=None, ctx=FAKE, k=4, B=2, hq=16, hkv=2, d=256, stream=None)
    a.update(kw)
    head = [a["kp"], a["vp"]] + ([a["ks"], a["vs"]] if fp8 else [])
    geom = [a["num"], a["table"], a["mp"], a["rows"]] + ([a["R"]] if fp8 else [])
    fn = lib.carat_paged_rope_append_fp8 if fp8 else lib.carat_paged_rope_append
    return fn(*head, *geom, a["kn"], a["vn"], a["kvs"], a["qo"], a["q"], a["qs"], a["cs"],
              a["trows"], a["r"], a["il"], a["pos"], a["cnt"], a["ctx"], a["k"], a["B"], a["hq"],
              a["hkv"], a["d"], a["stream"])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(kn=None), INVALID),
    (dict(vn=None), INVALID), (dict(cs=None), INVALID), (dict(ctx=None), INVALID),
    (dict(table=None), INVALID), (dict(q=None), INVALID), (dict(qo=None), INVALID),
    (dict(kp=MISALIGNED), INVALID), (dict(vp=MISALIGNED), INVALID), (dict(kn=MISALIGNED), INVALID),
    (dict(vn=MISALIGNED), INVALID), (dict(q=MISALIGNED), INVALID), (dict(qo=MISALIGNED), INVALID),
    (dict(cs=MISALIGNED), INVALID),
    (dict(num=0), INVALID), (dict(mp=0), INVALID), (dict(rows=64), INVALID),
    (dict(rows=130), INVALID), (dict(num=1 << 24), INVALID), (dict(mp=1 << 24), INVALID),
    (dict(kvs=504), INVALID), (dict(kvs=516), INVALID), (dict(qs=4088), INVALID),
    (dict(qs=4100), INVALID), (dict(trows=0), INVALID), (dict(r=0), INVALID), (dict(r=24), INVALID),
    (dict(r=272), INVALID), (dict(k=0), INVALID), (dict(k=513), INVALID), (dict(B=-1), INVALID),
    (dict(hq=-1), INVALID), (dict(hkv=0), INVALID), (dict(d=8, r=16), INVALID),
    (dict(d=264, r=16, kvs=4096, qs=8192), INVALID),
    (dict(d=144, r=16), UNSUPPORTED), (dict(d=1056, r=16, kvs=4096, qs=32768), UNSUPPORTED),
    (dict(d=2048, r=16, kvs=4096, qs=32768), UNSUPPORTED),
    (dict(B=1 << 30), INVALID),
    (dict(B=0), OK),
])
def test_rope_append_checks(lib, fp8, kw, status):
    assert _rope(lib, fp8, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(R=0), INVALID), (dict(R=8), INVALID),
    (dict(R=48), INVALID), (dict(R=256), INVALID),
])
def test_rope_append_fp8_checks(lib, kw, status):
    assert _rope(lib, True, **kw) == status


def _attn(lib, **kw):
    a = dict(out=FAKE, q=FAKE, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, num=8, table=FAKE, mp=4,
             rows=128, R=16, ctx=FAKE, k=4, B=2, hq=16, hkv=2, d=512, window=0, scale=0.1, ws=FAKE,
             wsb=0, stream=None)
    a.update(kw)
    return lib.carat_paged_verify_attention_fp8(
        a["out"], a["q"], a["kp"], a["vp"], a["ks"], a["vs"], a["num"], a["table"], a["mp"],
        a["rows"], a["R"], None, a["ctx"], a["k"], a["B"], a["hq"], a["hkv"], a["d"], a["window"],
        a["scale"], a["ws"], a["wsb"], a["stream"])


@pytest.mark.parametrize("kw,status", [
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(kp=None), INVALID),
    (dict(vp=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID),
    (dict(table=None), INVALID), (dict(ctx=None), INVALID), (dict(out=MISALIGNED), INVALID),
    (dict(q=MISALIGNED), INVALID), (dict(kp=MISALIGNED), INVALID), (dict(vp=MISALIGNED), INVALID),
    (dict(num=0), INVALID), (dict(mp=0), INVALID), (dict(rows=100), INVALID), (dict(R=24), INVALID),
    (dict(k=0), INVALID), (dict(k=17), INVALID), (dict(B=-1), INVALID), (dict(hq=15), INVALID),
    (dict(hq=0), INVALID), (dict(hkv=0), INVALID), (dict(window=-1), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(d=128), UNSUPPORTED), (dict(d=384), UNSUPPORTED), (dict(hq=65, hkv=1, k=1), UNSUPPORTED),
    (dict(hq=33, hkv=1, k=4), UNSUPPORTED), (dict(B=1 << 20), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws=MISALIGNED, wsb=1 << 40), WORKSPACE),
    (dict(wsb=16), WORKSPACE), (dict(B=0), OK),
])
def test_attention_checks(lib, kw, status):
    assert _attn(lib, **kw) == status


def test_workspace_query(lib):
    f = lib.carat_paged_fp8_workspace_bytes
    assert f(0, 1, 16, 2, 512, 1024) == 0
    assert f(2, 4, 16, 2, 128, 1024) == 0
    assert f(2, 17, 16, 2, 512, 1024) == 0
    assert f(2, 4, 16, 2, 512, 3) == 0
    a, b = f(2, 4, 16, 2, 512, 1024), f(64, 4, 16, 2, 512, 1024)
    assert 0 < a <= b


def test_bf16_paged_attention_checks(lib):
    def call(**kw):
        a = dict(out=FAKE, q=FAKE, kp=FAKE, vp=FAKE, num=8, table=FAKE, mp=4, rows=128, ctx=FAKE,
                 k=4, B=2, hq=16, hkv=2, d=512, scale=0.1, ws=FAKE, wsb=0, stream=None)
        a.update(kw)
        return lib.carat_global_verify_attention_paged(
            a["out"], a["q"], a["kp"], a["vp"], a["num"], a["table"], a["mp"], a["rows"], a["ctx"],
            a["k"], a["B"], a["hq"], a["hkv"], a["d"], a["scale"], a["ws"], a["wsb"], a["stream"])
    assert call(table=None) == INVALID
    assert call(rows=64) == INVALID
    assert call(q=None) == INVALID
    assert call(d=128) == UNSUPPORTED
    assert call(k=17) == INVALID
    assert call() == WORKSPACE
    assert call(B=0) == OK
