"""Refusals of the serving-step calls (kq8_write_kv, kq8_read_kv, kq8_tree_attn,
kq8_tree_commit, kq8_prompt_attn) that need no GPU: every bad argument is turned down
before anything is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from query_decode_attention_gb300 import build
    build.build()
    from query_decode_attention_gb300 import kq8
    return kq8


def _cache(lib, **kw):
    c = dict(k=256, v=256, kscale=256, vscale=256, num_pages=4, kv_bs=32, num_kv_heads=8,
             head_dim=128)
    c.update(kw)
    return lib.kq8_cache_t(*[c[n] for n in ("k", "v", "kscale", "vscale", "num_pages", "kv_bs",
                                            "num_kv_heads", "head_dim")])


# fake addresses: a call that is refused (or has nothing to do) touches none of them
def _rows(fn, lib, cache=None, bits=8, k=256, v=256, dtype=2, st=(1024, 128, 1024, 128), slot=256,
          T=4, status=None):
    return fn(ctypes.byref(cache or _cache(lib)), bits, k, v, dtype, *st, slot, T, status, None)


@pytest.mark.parametrize("name", ["kq8_write_kv", "kq8_read_kv"])
def test_rows_refusals(lib, name):
    fn = getattr(lib._lib, name)
    bad, un = lib.KQ8_ERR_INVALID_ARG, lib.KQ8_ERR_UNSUPPORTED
    assert _rows(fn, lib, T=0) == lib.KQ8_OK
    assert _rows(fn, lib, T=0, k=None, slot=None) == lib.KQ8_OK
    assert _rows(fn, lib, T=-1) == bad
    assert _rows(fn, lib, bits=2) == un
    assert _rows(fn, lib, dtype=3) == un
    assert _rows(fn, lib, dtype=-1) == un
    assert _rows(fn, lib, cache=_cache(lib, head_dim=64)) == un
    assert _rows(fn, lib, cache=_cache(lib, kv_bs=48)) == un
    assert _rows(fn, lib, cache=_cache(lib, num_kv_heads=70000)) == un
    assert _rows(fn, lib, cache=_cache(lib, kscale=8)) == bad
    for kw in (dict(k=None), dict(v=None), dict(slot=None), dict(k=257), dict(v=255),
               dict(slot=258), dict(status=258), dict(k=258, dtype=0),
               dict(st=(1 << 32, 128, 1024, 128)), dict(st=(1024, 128, 1024, (1 << 64) - 128))):
        assert _rows(fn, lib, **kw) == bad, kw


def test_a_read_refuses_overlapping_rows(lib):
    fn, bad = lib._lib.kq8_read_kv, lib.KQ8_ERR_INVALID_ARG
    for st in ((0, 128, 1024, 128), (1024, 0, 1024, 128), (1024, 127, 1024, 128),
               (1024, 128, 1023, 128), (1024, 128, 128, 511), (64, 4096, 1024, 128)):
        assert _rows(fn, lib, st=st) == bad, st


def test_a_read_refuses_k_rows_over_v_rows(lib):
    """k and v of 4 tokens x 8 heads: the same rows, rows that touch, and rows that lie
    among each other with other strides.  (What is apart is read on the GPU.)"""
    fn, bad = lib._lib.kq8_read_kv, lib.KQ8_ERR_INVALID_ARG
    k = 1 << 20
    for d, st in ((0, (1024, 128)), (64, (1024, 128)), (1024 * 3, (1024, 128)),
                  (1024 * 3 + 127, (1024, 128)), (256, (4096, 256)), (127, (4096, 256)),
                  (4096 * 3 + 256 * 7 + 127, (4096, 256)), (128, (128, 512)), (128 * 3, (128, 512))):
        for a, b in ((k, k + 2 * d), (k + 2 * d, k)):
            assert _rows(fn, lib, k=a, v=b, st=st + st) == bad, (d, st)
    assert _rows(fn, lib, k=k, v=k + 2 * 128, st=(2048, 256, 2048, 128)) == bad


def _tree(lib, cache=None, dtype=2, qs=(2048, 128), total_q=8, max_pages=2, mask=256, words=1,
          max_seq_len=64, max_q_len=8, B=1, nq=16, ws=512, ws_bytes=1 << 30, out=1 << 30, q=256,
          pt=256, sl=256, qo=256):
    return lib._lib.kq8_tree_attn(out, q, dtype, *qs, total_q, ctypes.byref(cache or _cache(lib)),
                                  pt, max_pages, sl, qo, mask, words, max_seq_len, max_q_len, B,
                                  nq, 0.1, ws, ws_bytes, None)


def test_tree_refusals(lib):
    bad, un, ws = lib.KQ8_ERR_INVALID_ARG, lib.KQ8_ERR_UNSUPPORTED, lib.KQ8_ERR_WORKSPACE
    assert _tree(lib, B=0) == lib.KQ8_OK
    assert _tree(lib, max_q_len=0) == lib.KQ8_OK
    for kw in (dict(cache=_cache(lib, head_dim=64)), dict(dtype=3), dict(nq=12), dict(nq=72),
               dict(B=65536), dict(max_q_len=1025, max_seq_len=2048, max_pages=64, words=33)):
        assert _tree(lib, **kw) == un, kw
    for kw in (dict(B=-1), dict(total_q=-1), dict(max_q_len=-1), dict(words=-1),
               dict(max_seq_len=65), dict(max_q_len=33, words=2, max_seq_len=32),
               dict(max_q_len=33, words=1), dict(out=None), dict(q=None), dict(sl=None),
               dict(qo=None), dict(pt=None), dict(q=260), dict(out=(1 << 30) + 2), dict(q=264, dtype=0),
               dict(out=256), dict(out=256 + 2 * 8 * 2048 - 8), dict(q=(1 << 30) + 8),
               dict(qs=(2046, 128)), dict(qs=(2048, 130)), dict(qs=(1 << 40, 128)),
               dict(mask=258)):
        assert _tree(lib, **kw) == bad, kw
    for kw in (dict(ws=None), dict(ws=512 + 64), dict(ws_bytes=1024)):
        assert _tree(lib, **kw) == ws, kw


def test_tree_workspace(lib):
    f = lib.kq8_tree_workspace_bytes
    assert f(-1, 16, 8, 64, 8) == 0 and f(1, 12, 8, 64, 8) == 0 and f(1, 16, 8, -1, 8) == 0
    assert f(0, 16, 8, 0, 0) >= 256
    one = f(1, 16, 8, 4096, 8)
    assert one % 256 == 0 and f(4, 16, 8, 4096, 8) >= one
    # partials stay bounded however many and long the sequences are
    for B, nq, nkv, n, nodes in ((65535, 64, 8, 1 << 20, 256), (512, 64, 8, 131072, 1024),
                                 (1, 8, 1, (1 << 29) - 1, 1024)):
        assert f(B, nq, nkv, n, nodes) <= 1 << 30


def _commit(lib, cache=None, bits=8, pt=256, max_pages=2, base=256, path=256, plen=256, max_path=4,
            B=1, status=None):
    return lib._lib.kq8_tree_commit(ctypes.byref(cache or _cache(lib)), bits, pt, max_pages, base,
                                    path, plen, max_path, B, status, None)


def test_commit_refusals(lib):
    bad, un = lib.KQ8_ERR_INVALID_ARG, lib.KQ8_ERR_UNSUPPORTED
    assert _commit(lib, B=0) == lib.KQ8_OK
    assert _commit(lib, max_path=0) == lib.KQ8_OK
    for kw in (dict(bits=3), dict(B=65536), dict(max_pages=1 << 25),
               dict(cache=_cache(lib, head_dim=32))):
        assert _commit(lib, **kw) == un, kw
    for kw in (dict(B=-1), dict(max_path=-1), dict(max_pages=-1), dict(pt=None), dict(base=None),
               dict(path=None), dict(plen=None), dict(status=257)):
        assert _commit(lib, **kw) == bad, kw


def _prompt(lib, out=1 << 30, q=256, k=256, v=256, dtype=2, st=(4096, 128) * 3, cu=256, total=64,
            max_len=64, B=1, nq=16, nkv=8, scale=0.1, status=None):
    return lib._lib.kq8_prompt_attn(out, q, k, v, dtype, *st, cu, total, max_len, B, nq, nkv, scale,
                                    status, None)


def test_prompt_refusals(lib):
    bad, un = lib.KQ8_ERR_INVALID_ARG, lib.KQ8_ERR_UNSUPPORTED
    for kw in (dict(B=0), dict(max_len=0), dict(total=0)):
        assert _prompt(lib, **kw) == lib.KQ8_OK, kw
    for kw in (dict(dtype=0), dict(dtype=3), dict(nq=12), dict(nq=72), dict(B=65536),
               dict(nq=70000, nkv=70000)):
        assert _prompt(lib, **kw) == un, kw
    for kw in (dict(B=-1), dict(total=-1), dict(max_len=-1), dict(nq=0), dict(nkv=0),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(out=None), dict(q=None), dict(k=None), dict(v=None),
               dict(cu=None), dict(out=(1 << 30) + 8), dict(out=256),
               dict(q=(1 << 30) + 2 * 2048 * 64 - 16), dict(k=(1 << 30) - 2 * 64 * 4096 + 8192),
               dict(v=1 << 30), dict(q=264), dict(k=258), dict(v=264),
               dict(st=(4100, 128) * 3), dict(st=(4096, 128, 4096, 132, 4096, 128)),
               dict(st=(4096, 128, 4096, 128, 1 << 40, 128)), dict(status=257)):
        assert _prompt(lib, **kw) == bad, kw


def test_binding_refuses_host_and_misshapen_tensors(lib):
    torch = pytest.importorskip("torch")
    t = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        lib.kq8_prompt_attn(t, t, t, t, torch.zeros(2, dtype=torch.int32), 4, 0.1)
    cache = lib.PagedKVCache(1, 8, 32, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        lib.kq8_write_kv(cache, t, t, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="q8 cache"):
        lib.kq8_tree_attn(t, t, lib.PagedKVCache(1, 8, 32, device="cpu", bits=4), None, None, None,
                          None, 4, 4, 0.1, None)
