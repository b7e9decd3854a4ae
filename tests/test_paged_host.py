"""Refusals of the paged entry points, found on the host before anything is enqueued (no
compute call runs here), and the binding's own checks."""
import ctypes

import pytest
import torch

FAKE = 1 << 20          # aligned, never dereferenced: the calls fail their checks first


def _cache(tam, **kw):
    f = dict(k_pages=FAKE, v_pages=FAKE, k_scale=None, v_scale=None, n_pages=8,
             page_stride=16 * 2 * 64, row_stride=2 * 64, head_stride=64, page_size=16, Hkv=2, d=64,
             dtype=tam.TAM_BF16)
    f.update(kw)
    return tam._KvCacheStruct(**f)


def _batch(tam, **kw):
    f = dict(page_table=FAKE, cu_rows=FAKE, kv_len=FAKE, n_seq=3, max_pages=4, max_rows=0)
    f.update(kw)
    return tam._PagedBatchStruct(**f)


def _calls(tam, kv, b, T=5, Hq=4, dtype=0, p=FAKE, ws=FAKE, nbytes=1 << 40):
    L = tam.lib()
    kv = ctypes.addressof(kv) if kv is not None else None
    b = ctypes.addressof(b) if b is not None else None
    return [L.tam_kv_cache_write(T, dtype, p, p, kv, b, ws, nbytes, None),
            L.tam_kv_cache_read(T, dtype, p, p, kv, b, ws, nbytes, None),
            L.tam_paged_gqa_attention(T, Hq, dtype, p, kv, b, p, None, ws, nbytes, None)]


def test_every_call_refuses_a_bad_cache_or_batch(tam_lib):
    T = tam_lib
    bad, uns = T.TAM_ERR_INVALID_ARG, T.TAM_ERR_UNSUPPORTED
    for kw, rc in [
            (dict(k_pages=None), bad), (dict(v_pages=None), bad), (dict(k_pages=FAKE + 8), bad),
            (dict(dtype=7), bad), (dict(n_pages=0), bad), (dict(Hkv=0), bad),
            (dict(page_size=0), bad), (dict(page_size=8), uns), (dict(page_size=48), uns),
            (dict(page_size=512), uns), (dict(d=96), uns), (dict(n_pages=1 << 31), uns),
            (dict(row_stride=0), bad), (dict(head_stride=63), bad), (dict(page_stride=-64), bad),
            (dict(row_stride=132), bad), (dict(page_stride=1 << 40), uns),
            (dict(dtype=T.TAM_E4M3), bad),                                       # no scales
            (dict(dtype=T.TAM_E4M3, k_scale=FAKE, v_scale=FAKE + 1), bad)]:
        assert _calls(T, _cache(T, **kw), _batch(T)) == [rc] * 3, kw
    for kw, rc in [(dict(page_table=None), bad), (dict(cu_rows=None), bad), (dict(kv_len=None), bad),
                   (dict(n_seq=0), bad), (dict(max_pages=0), bad), (dict(max_rows=-1), bad),
                   (dict(n_seq=32769), uns), (dict(max_pages=1 << 27), uns)]:
        assert _calls(T, _cache(T), _batch(T, **kw)) == [rc] * 3, kw
    assert _calls(T, None, _batch(T)) == [bad] * 3
    assert _calls(T, _cache(T), None) == [bad] * 3


def test_every_call_refuses_bad_rows_and_workspaces(tam_lib):
    T = tam_lib
    kv, b = _cache(T), _batch(T)
    bad, uns = T.TAM_ERR_INVALID_ARG, T.TAM_ERR_UNSUPPORTED
    assert _calls(T, kv, b, T=-1) == [bad] * 3
    assert _calls(T, kv, b, T=1 << 31) == [uns] * 3
    assert _calls(T, kv, b, dtype=T.TAM_E4M3) == [bad] * 3
    assert _calls(T, kv, b, dtype=T.TAM_F32) == [uns] * 3          # fp32 rows, bf16 cache
    assert _calls(T, kv, b, p=None) == [bad] * 3
    assert _calls(T, kv, b, p=FAKE + 4) == [bad] * 3
    assert _calls(T, kv, b, ws=None) == [bad] * 3
    assert _calls(T, kv, b, ws=FAKE + 4) == [bad] * 3
    assert _calls(T, kv, b, nbytes=255) == [T.TAM_ERR_WORKSPACE] * 3
    L = T.lib()
    for Hq, rc in ((3, bad), (0, bad), (2 * 129, uns)):
        assert _calls(T, kv, b, Hq=Hq)[2] == rc
        assert L.tam_paged_attention_workspace(5, Hq, 0, ctypes.addressof(kv),
                                               ctypes.addressof(b)) == 0
    n = L.tam_paged_attention_workspace(5, 4, 0, ctypes.addressof(kv), ctypes.addressof(b))
    assert n > 0 and n % 256 == 0
    assert _calls(T, kv, b, nbytes=n - 1)[2] == T.TAM_ERR_WORKSPACE


def test_binding_refuses_host_caches(tam_lib):
    z = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tam_lib.PagedKVCache(z, z)


def test_workspace_that_a_graph_holds_is_not_freed_when_it_grows(tam_lib):
    ws = tam_lib.Workspace("cpu")
    a = ws.get(1000)
    ws.captured = True
    b = ws.get(5000)
    assert b.numel() >= 5000 and ws._kept[0] is a and not ws.captured
    assert ws.get(10) is b


def test_binding_refuses_workspaces_and_streams_of_another_device(tam_lib):
    """Before the call touches the device: its memory would not be reachable, or not ordered."""
    import types
    dev = torch.device("cuda:0")
    here = types.SimpleNamespace(device=dev)
    held = tam_lib.Workspace("cpu")
    held.get(1000)

    def body(handle, get_ws):
        raise AssertionError("the call went on")

    other = types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    for kw in (dict(workspace=held), dict(workspace=tam_lib.Workspace("cpu")),
               dict(workspace=tam_lib.Workspace("cuda:1")), dict(stream=other)):
        with pytest.raises(ValueError, match="cache's CUDA device"):
            tam_lib._paged_call(here, here, (), kw.get("workspace"), kw.get("stream"), False, body)


def test_default_workspaces_of_many_streams_are_bounded(tam_lib, monkeypatch):
    import types
    here = types.SimpleNamespace(device=torch.device("cuda:0"))
    kept = {}
    monkeypatch.setattr(tam_lib, "_paged_ws", types.SimpleNamespace())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for i in range(100):
        monkeypatch.setattr(tam_lib, "_stream_handle", lambda index: 1000 + i)
        for _ in range(2):
            tam_lib._paged_call(here, here, (), None, None, False, lambda handle, get_ws: (handle, None))
            ws = tam_lib._paged_ws.__dict__[0, 1000 + i]
            assert kept.setdefault(i, ws) is ws                # a stream keeps its own
    assert len(tam_lib._paged_ws.__dict__) == 16
