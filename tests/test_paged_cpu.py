"""The paged cache and cross attention without a GPU: the oracle against torch in fp64, and the refusals of
the C entries and of the binding (no kernel is launched)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_sparse_video_int8_b200 as bsva
from oracle import paged

P = ctypes.c_void_p(0x10000)
F0 = ctypes.c_float(0)


def _cache(**kw):
    d = dict(n_pages=8, page_size=16, H=2, d=128, dtype=0, k=0x10000, v=0x10000, k_scale=0x10000, v_scale=0x10000)
    d.update(kw)
    return bsva.PagedKVStruct(**d)


def _batch(**kw):
    d = dict(S=2, T=5, max_q=4, max_kv=64, max_pages=4, q_start=0x10000, kv_len=0x10000, page_table=0x10000)
    d.update(kw)
    return bsva.PagedBatchStruct(**d)


def _write(c, b, k=P, v=P, ks=256, vs=256, ws=P, n=256):
    return bsva.load().bsva_paged_kv_write(ctypes.byref(c) if c else None, ctypes.byref(b) if b else None, k, v, ks, vs,
                                           ws, n, None)


def _read(c, b, first=None, L=64, ko=P, vo=P, ws=P, n=256):
    return bsva.load().bsva_paged_kv_read(ctypes.byref(c), ctypes.byref(b), first, L, ko, vo, ws, n, None)


def _attend(c, b, q=P, stride=512, Hq=4, causal=1, window=0, scale=F0, out=P, lse=None, ws=P, n=1 << 30):
    return bsva.load().paged_attn_fwd(ctypes.byref(c), ctypes.byref(b), q, stride, Hq, causal, window, scale, out, lse,
                                      ws, n, None)


def _error():
    return bsva.load().bsva_last_error().decode()


# ------------------------------------------------------------------------------------------- the oracle
def test_row_quantiser_hand_cases():
    c, s = paged.quantize_rows(np.array([[127, -127, 0.5, 1.5, 2.5, -0.5]], np.float32))
    assert s[0] == 1 and c[0].tolist() == [127, -127, 0, 2, 2, 0]     # ties go to the even code
    c, s = paged.quantize_rows(np.zeros((1, 4), np.float32))
    assert s[0] == 0 and not c.any()
    c, s = paged.quantize_rows(np.array([[1e-40, -1e-40, 0, 5e-41]], np.float32))
    assert c[0].tolist() == [127, -127, 0, 64] or c[0].tolist() == [127, -127, 0, 63]
    x = np.random.default_rng(0).standard_normal((50, 64)).astype(np.float32)
    c, s = paged.quantize_rows(x)
    assert np.abs(paged.dequantize_rows(c, s) - x).max() <= s.max() * (0.5 + 1e-5)


@pytest.mark.parametrize("n,kv,causal,window", [(1, 1, True, 0), (5, 5, True, 0), (3, 9, True, 0), (4, 12, True, 3),
                                                (4, 7, False, 0), (6, 4, True, 0)])
def test_oracle_attention_against_sdpa(n, kv, causal, window):
    g = torch.Generator().manual_seed(n * 100 + kv)
    q, k, v = (torch.randn((x, 16), dtype=torch.float64, generator=g) for x in (n, kv, kv))
    ok = paged.visible(n, kv, causal, window)
    for i in range(n):       # the definition, one comparison at a time
        p = kv - n + i
        assert ok[i].tolist() == [(not causal or t <= p) and (not window or t > p - window) for t in range(kv)]
    o, lse, _ = paged.attention_rows(q.numpy(), k.numpy(), v.numpy(), ok)
    live = ok.any(1)
    ref = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], v[None], torch.from_numpy(ok)[None])[0]
    assert np.allclose(o[live], ref.numpy()[live], atol=1e-12)
    assert np.allclose(lse[live], torch.logsumexp((q @ k.T / 4).masked_fill(~torch.from_numpy(ok), -math.inf), 1)
                       .numpy()[live], atol=1e-12)
    assert (o[~live] == 0).all() and (lse[~live] == -np.inf).all()


# ------------------------------------------------------------------------------------------- refusals
@pytest.mark.parametrize("bad,code,word", [
    (dict(d=96), 2, "head dim"), (dict(page_size=24), 1, "page_size"), (dict(page_size=8), 1, "page_size"),
    (dict(page_size=512), 1, "page_size"), (dict(n_pages=0), 1, "n_pages"), (dict(H=0), 1, "H ="),
    (dict(dtype=2), 1, "dtype"), (dict(n_pages=2 ** 30, H=1, page_size=16), 1, "below 2^31"),
    (dict(n_pages=2 ** 24, H=8, page_size=16), 1, "below 2^31"), (dict(k=None), 1, "NULL"), (dict(v=0x10008), 1, "aligned"),
    (dict(k_scale=None), 1, "NULL"), (dict(v_scale=0x10002), 1, "aligned")])
def test_bad_caches_are_refused(bad, code, word):
    c = _cache(**bad)
    for f in (_write, _read, _attend):
        assert f(c, _batch()) == code and word in _error()
    if not {"k", "v", "k_scale", "v_scale"} & set(bad):
        assert bsva.load().bsva_paged_workspace_bytes(ctypes.byref(c), ctypes.byref(_batch()), 4) == 0


@pytest.mark.parametrize("bad,word", [
    (dict(S=0), "S ="), (dict(S=65536), "S ="), (dict(T=-1), "T ="), (dict(max_q=0), "max_q"),
    (dict(max_kv=0), "max_kv"), (dict(max_kv=65), "max_pages"), (dict(max_pages=0), "max_pages"),
    (dict(kv_len=None), "NULL"), (dict(page_table=None), "NULL"), (dict(page_table=0x10001), "aligned")])
def test_bad_batches_are_refused(bad, word):
    for f in (_write, _read, _attend):
        assert f(_cache(), _batch(**bad)) == 1 and word in _error()


def test_bad_arguments_are_refused():
    c, b = _cache(), _batch()
    assert _write(None, b) == 1 and _write(c, None) == 1
    assert _write(c, _batch(q_start=None)) == 1 and "NULL" in _error()
    for kw in (dict(ks=248), dict(vs=260), dict(ks=-256)):
        assert _write(c, b, **kw) == 1 and "stride" in _error()
    assert _write(c, b, k=None) == 1 and _write(c, b, v=ctypes.c_void_p(0x10002)) == 1
    assert _write(c, b, n=128) == 3 and _write(c, b, ws=None) == 3 and _write(c, b, ws=ctypes.c_void_p(0x10010)) == 3
    assert _read(c, b, L=0) == 1 and "L =" in _error()
    assert _read(c, b, ko=None) == 1 and _read(c, b, first=ctypes.c_void_p(0x10001)) == 1 and _read(c, b, n=0) == 3
    for kw, word in ((dict(Hq=3), "multiple"), (dict(Hq=0), "multiple"), (dict(stride=500), "stride"),
                     (dict(stride=508), "stride"), (dict(causal=2), "causal"), (dict(window=-1), "window"),
                     (dict(window=4, causal=0), "window"), (dict(scale=ctypes.c_float(math.nan)), "finite"),
                     (dict(scale=ctypes.c_float(math.inf)), "finite"), (dict(q=None), "NULL"),
                     (dict(out=ctypes.c_void_p(0x10008)), "aligned"), (dict(lse=ctypes.c_void_p(0x10002)), "aligned")):
        assert _attend(c, b, **kw) == 1 and word in _error(), kw
    need = bsva.load().bsva_paged_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 4)
    assert need >= 256
    assert _attend(c, b, n=need - 1) == 3 and "workspace" in _error()


def test_workspace_holds_the_splits_of_any_window():
    # 2 sequences of 1 token over up to 131072 keys, 1 key head: many splits of partial rows (d + 2 floats)
    c, b = _cache(H=1, n_pages=8192, page_size=16), _batch(S=2, T=2, max_q=1, max_kv=131072, max_pages=8192)
    n = bsva.load().bsva_paged_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 8)
    assert n >= 256 + 2 * (2 * 8 * 130 * 4)
    last = 0
    for kv in range(1, 20000, 37):
        b.max_kv = kv
        m = bsva.load().bsva_paged_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 8)
        assert m >= last         # more keys never need less, so a window's fewer keys always fit
        last = m


def test_cross_attention_refusals():
    lib = bsva.load()

    def call(s, Hkv=2, q=P, k=P, v=P, kl=None, scale=F0, out=P, lse=None, ws=P, n=1 << 30):
        return lib.cross_attn_fwd(s, Hkv, q, k, v, kl, scale, out, lse, ws, n, None)
    s = bsva.Shape(2, 4, 100, 77, 64, 0)
    assert call(bsva.Shape(2, 4, 100, 0, 64, 0)) == 1 and call(bsva.Shape(2, 4, 100, 77, 80, 0)) == 2
    assert call(s, Hkv=3) == 1 and "multiple" in _error()
    assert call(s, q=None) == 1 and call(s, v=ctypes.c_void_p(0x10004)) == 1 and call(s, kl=ctypes.c_void_p(0x10001)) == 1
    assert call(s, scale=ctypes.c_float(math.nan)) == 1 and call(s, n=64) == 3
    assert lib.bsva_cross_attn_workspace_bytes(s, 3) == 0 and lib.bsva_cross_attn_workspace_bytes(s, 2) >= 256


def test_binding_refuses_cpu_tensors_and_bad_types():
    t = torch.zeros((2, 2, 16, 64), dtype=torch.int8)
    with pytest.raises(ValueError, match="CUDA"):
        bsva.PagedKVCache.over(t, t)
    with pytest.raises(TypeError):
        bsva.PagedKVCache.over(t.float(), t.float())
    with pytest.raises(TypeError):
        bsva.PagedKVCache(4, 16, 2, 64, dtype=torch.float16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        bsva.PagedBatch(i, i[:2], i[:2, None], 1, 16)
    x = torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bsva.cross_attn_fwd(x, x, x)


@pytest.mark.parametrize("device,want", [(None, "cuda"), (0, 0), (1, 1), ("cuda:0", "cuda:0")])
def test_a_cache_is_allocated_on_the_device_it_is_given(monkeypatch, device, want):
    class Seen(Exception):
        pass

    def zeros(*a, device=None, **kw):
        raise Seen(device)
    monkeypatch.setattr(torch, "zeros", zeros)
    with pytest.raises(Seen) as e:
        bsva.PagedKVCache(4, 16, 2, 64, device=device)
    assert e.value.args == (want,)
