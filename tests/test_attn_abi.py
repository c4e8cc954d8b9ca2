"""The attention and key/value cache calls refuse bad arguments on the host, before any launch
(no GPU here), the binding's constants match the header, and the validation runs clean under
AddressSanitizer and UndefinedBehaviorSanitizer (host code only, launchers stubbed)."""
import ctypes
import os
import re
import subprocess

import pytest

import microscaling_quantized_convolution_amd as mq

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
S0 = ctypes.c_void_p(0)
OK, ARG, SHAPE = mq.MQ_OK, mq.MQ_ERR_ARG, mq.MQ_ERR_SHAPE
UNSUPPORTED, WORKSPACE = mq.MQ_ERR_UNSUPPORTED, mq.MQ_ERR_WORKSPACE


def cache(pages=8, page=32, heads=2, dim=64, k=0x1000, v=0x2000, ks=0x3000, vs=0x4000):
    return mq.mq_kv_cache(pages, page, heads, dim, k, v, ks, vs)


def rows(tokens=4, heads=2, dim=64, dtype=mq.MQ_BF16, data=0x10000, ts=None, hs=None):
    return mq.mq_rows(data, heads * dim if ts is None else ts, dim if hs is None else hs, tokens,
                      heads, dim, dtype)


def test_header_constants_match_binding():
    hdr = open(os.path.join(ROOT, "include", "mq.h")).read()
    assert re.search(r"MQ_F16 = %d, MQ_BF16 = %d " % (mq.MQ_F16, mq.MQ_BF16), hdr)
    assert int(re.search(r"#define MQ_KV_BLOCK (\d+)", hdr).group(1)) == mq.MQ_KV_BLOCK


def test_append_refusals():
    def call(c=cache(), k=rows(), v=rows(), table=0x100, lens=0x200, cu=0x300, n=2, width=4):
        return mq.lib().mq_kv_append(c, k, v, table, lens, cu, n, width, S0)
    for bad in (dict(c=None), dict(k=None), dict(v=None), dict(table=None), dict(lens=None),
                dict(cu=None), dict(n=-1), dict(width=-1), dict(table=0x102), dict(lens=0x201),
                dict(c=cache(page=24)), dict(c=cache(page=0)), dict(c=cache(pages=0)),
                dict(c=cache(heads=0)), dict(c=cache(k=0)), dict(c=cache(vs=0)),
                dict(c=cache(v=0x2008)), dict(k=rows(dtype=3)), dict(k=rows(dtype=0)),
                dict(k=rows(tokens=-1)), dict(k=rows(data=0)), dict(v=rows(data=0x10008)),
                dict(v=rows(ts=132)), dict(k=rows(hs=-64)), dict(k=rows(ts=-128))):
        assert call(**bad) == ARG, bad
    for bad in (dict(k=rows(tokens=3)), dict(v=rows(heads=1)), dict(k=rows(dtype=mq.MQ_F16)),
                dict(c=cache(heads=4)), dict(c=cache(dim=128))):
        assert call(**bad) == SHAPE, bad
    odd = dict(c=cache(dim=80), k=rows(dim=80), v=rows(dim=80))
    assert call(**odd) == UNSUPPORTED
    assert call(width=1 << 26) == UNSUPPORTED  # positions past 2^30
    assert call(c=cache(pages=1 << 30)) == UNSUPPORTED  # 2^31 blocks and more
    # nothing to do is no error
    assert call(n=0, table=None, lens=None, cu=None) == OK
    assert call(k=rows(tokens=0, data=0), v=rows(tokens=0, data=0)) == OK
    assert call(width=0, table=None) == OK


def test_cached_refusals():
    need = mq.mq_attn_cached_workspace_bytes(2, 4, 2, 64, 2, 5000)
    assert need > 0

    def call(c=cache(), q=rows(heads=4), out=rows(heads=4), table=0x100, lens=0x200, n=2, width=400,
             q_len=2, max_len=5000, weights=None, ws=0x8000, size=need):
        return mq.lib().mq_attn_cached(c, q, out, table, lens, n, width, q_len, max_len, 0.1,
                                       weights, ws, size, S0)
    for bad in (dict(c=None), dict(q=None), dict(out=None), dict(table=None), dict(lens=None),
                dict(n=-2), dict(width=-1), dict(q_len=0), dict(max_len=-1), dict(weights=0x102),
                dict(ws=0x8008), dict(q=rows(heads=4, data=0)), dict(out=rows(heads=4, dtype=7)),
                dict(c=cache(page=8))):
        assert call(**bad) == ARG, bad
    for bad in (dict(q=rows(heads=3), out=rows(heads=3)), dict(out=rows(heads=2)), dict(q_len=1),
                dict(n=1), dict(c=cache(dim=128)), dict(out=rows(heads=4, dtype=mq.MQ_F16))):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(ws=None), dict(size=need - 1), dict(weights=0x100)):
        assert call(**bad) == WORKSPACE, bad
    assert call(max_len=(1 << 30) + 1) == UNSUPPORTED
    assert call(width=1 << 27) == UNSUPPORTED
    five = dict(c=cache(dim=80), q=rows(heads=4, dim=80), out=rows(heads=4, dim=80))
    assert call(**five) == UNSUPPORTED
    assert call(n=0, q=rows(heads=4, tokens=0, data=0), out=rows(heads=4, tokens=0, data=0)) == OK


def test_cached_workspace_bytes():
    need = mq.mq_attn_cached_workspace_bytes
    assert need(1, 8, 2, 64, 1, 300) == 0  # one launch, no parts
    assert need(1, 8, 2, 64, 1, 300, True) > 0
    assert need(4, 8, 2, 128, 1, 100000, True) > need(4, 8, 2, 128, 1, 100000) > 0
    for bad in ((0, 8, 2, 64, 1, 9), (1, 8, 3, 64, 1, 9), (1, 8, 2, 65, 1, 9), (1, 8, 2, 64, 0, 9),
                (1, 8, 2, 64, 1, -1), (1, 8, 0, 64, 1, 9), (1, 8, 2, 64, 1 << 30, 9)):
        assert need(*bad) == 0, bad


def test_prompt_refusals():
    def call(q=rows(heads=4), k=rows(), v=rows(), out=rows(heads=4), cu=0x100, n=2, max_len=4):
        return mq.lib().mq_attn_prompt(q, k, v, out, cu, n, max_len, 0.1, S0)
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(cu=None),
                dict(cu=0x101), dict(n=-1), dict(max_len=-1), dict(k=rows(data=0x10004)),
                dict(v=rows(dtype=0)), dict(q=rows(heads=0))):
        assert call(**bad) == ARG, bad
    for bad in (dict(k=rows(tokens=5)), dict(out=rows(heads=2)), dict(k=rows(heads=3), v=rows(heads=3)),
                dict(v=rows(heads=1)), dict(v=rows(dim=128)), dict(k=rows(dtype=mq.MQ_F16))):
        assert call(**bad) == SHAPE, bad
    assert call(max_len=(1 << 30) + 1) == UNSUPPORTED
    assert call(k=rows(ts=(1 << 24) + 8)) == UNSUPPORTED
    empty = rows(heads=4, tokens=0, data=0)
    none = rows(tokens=0, data=0)
    assert call(q=empty, k=none, v=none, out=empty) == OK
    assert call(n=0, cu=None) == OK and call(max_len=0) == OK


def test_evict_refusals():
    def call(c=cache(), w=0x100, table=0x200, lens=0x300, new=0x400, new_lens=0x500, kept=0x600,
             n=2, width=4, new_width=2, keep=40, recent=8):
        return mq.lib().mq_kv_evict(c, w, table, lens, new, new_lens, kept, n, width, new_width,
                                    keep, recent, S0)
    for bad in (dict(c=None), dict(w=None), dict(w=0x102), dict(table=None), dict(lens=None),
                dict(new=None), dict(new_lens=None), dict(kept=None), dict(n=-1), dict(width=-1),
                dict(new_width=-1), dict(keep=-1), dict(recent=-1), dict(new_lens=0x300),
                dict(kept=0x601)):
        assert call(**bad) == ARG, bad
    assert call(keep=65) == SHAPE
    assert call(c=cache(dim=72)) == UNSUPPORTED
    assert call(width=1 << 26) == UNSUPPORTED
    assert call(n=0, table=None, lens=None, new=None, new_lens=None, kept=None) == OK


@pytest.mark.skipif(not os.path.isdir("/opt/rocm/include"), reason="needs the HIP headers")
def test_host_validation_under_sanitizers(tmp_path):
    exe = str(tmp_path / "attn_asan")
    subprocess.check_call([
        "g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
        "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer",
        "-O1", "-g", os.path.join(HERE, "attn_asan_driver.cpp"),
        os.path.join(ROOT, "microscaling_quantized_convolution_amd", "csrc", "mq_attn_api.cpp"),
        "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "0 failures" in r.stdout and "runtime error" not in r.stderr
