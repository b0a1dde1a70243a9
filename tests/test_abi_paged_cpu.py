"""Host checks of the paged cache operators' C entry points and binding, without a GPU:
every call here is refused before anything is launched, or is an empty one."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def cmp():
    import streaming_kv_cache_varlen_b200 as m
    return m


P = 0x10000


def rope(cmp, **kw):
    d = dict(sin=P, cos=P, dim=64, pairs=0, dtype=0)
    d.update(kw)
    return ctypes.byref(cmp.cmp_rope(*(d[k] for k in ("sin", "cos", "dim", "pairs", "dtype"))))


def norm(cmp, args=None, r=None, eps=1e-6, dtype=1, **kw):
    d = dict(T=0, Hq=8, Hk=2, D=128, q_stride=1024, k_stride=256, q_out_stride=1024, k_out_stride=256)
    d.update(kw)
    a = dict(q=P, k=P, qw=P, kw=P, qo=2 * P, ko=2 * P)
    a.update(args or {})
    return cmp.lib.cmp_qk_norm_rope(a["q"], a["k"], a["qw"], a["kw"], r, eps, dtype, a["qo"], a["ko"], None,
                                    ctypes.byref(cmp.cmp_qk_dims(**d)))


def test_norm_refusals(cmp):
    assert norm(cmp) == 0                                         # T == 0: nothing to do
    assert cmp.lib.cmp_qk_norm_rope(P, P, P, P, None, 1e-6, 1, P, P, None, None) == 1
    assert norm(cmp, dtype=2) == 3
    for kw in (dict(Hq=0), dict(Hq=1025), dict(Hk=-1), dict(Hk=1025), dict(D=8), dict(D=100), dict(D=272), dict(T=-1),
               dict(q_stride=1023), dict(q_stride=1020), dict(k_stride=248), dict(q_out_stride=512), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf"))):
        assert norm(cmp, **kw) == 2, kw
    for name in ("q", "k", "qw", "kw", "qo", "ko"):
        assert norm(cmp, {name: None}, T=4) == 1, name
        assert norm(cmp, {name: P + 8}, T=4) == 2, name
    assert norm(cmp, dict(q=P, qo=P), T=4, q_stride=2048) == 2     # in place with another stride
    for bad, st in ((dict(dim=8), 2), (dict(dim=24), 2), (dict(dim=144), 2), (dict(pairs=2), 3), (dict(dtype=2), 3),
                    (dict(sin=None), 1), (dict(cos=None), 1), (dict(sin=P + 4), 2)):
        assert norm(cmp, r=rope(cmp, **bad), T=4) == st, bad


def append(cmp, args=None, r=None, eps=1e-6, dtype=1, **kw):
    d = dict(B=2, T=4, Hk=2, D=128, k_stride=256, v_stride=256, block_num=8, page_size=16, table_stride=4)
    d.update(kw)
    a = dict(k=P, v=P, w=P, tbl=P, cu=P, sp=P, kc=P, vc=P)
    a.update(args or {})
    return cmp.lib.cmp_kv_append(a["k"], a["v"], a["w"], r, eps, a["tbl"], a["cu"], a["sp"], dtype, a["kc"], a["vc"],
                                 None, ctypes.byref(cmp.cmp_kv_dims(**d)))


def test_append_refusals(cmp):
    assert append(cmp, T=0) == 0 and append(cmp, B=0, T=0) == 0
    assert cmp.lib.cmp_kv_append(P, P, None, None, 1e-6, P, P, P, 1, P, P, None, None) == 1
    assert append(cmp, dtype=7) == 3
    for kw in (dict(B=-1), dict(B=0), dict(T=-1), dict(Hk=0), dict(Hk=257), dict(D=24), dict(D=0), dict(k_stride=255),
               dict(v_stride=128), dict(page_size=0), dict(page_size=1025), dict(block_num=0),
               dict(block_num=2 ** 31 // 16), dict(table_stride=0), dict(eps=-1e-6)):
        assert append(cmp, **kw) == 2, kw
    for name in ("k", "v", "tbl", "cu", "kc", "vc"):
        assert append(cmp, {name: None}) == 1, name
    for name in ("k", "v", "w", "kc", "vc"):
        assert append(cmp, {name: P + 8}) == 2, name
    for name in ("tbl", "cu", "sp"):
        assert append(cmp, {name: P + 2}) == 2, name
    assert append(cmp, r=rope(cmp, dim=144)) == 2


def attn(cmp, args=None, scale=0.1, window=0, kb=1, ks=1, dtype=1, ws_bytes=1 << 40, **kw):
    d = dict(B=2, T=4, Hq=8, Hk=2, D=128, q_stride=1024, block_num=8, page_size=16, table_stride=4, max_len=0)
    d.update(kw)
    a = dict(q=P, kc=P, vc=P, tbl=P, cu=P, sp=P, out=P, lse=P, ws=P)
    a.update(args or {})
    return cmp.lib.cmp_paged_attention(a["q"], a["kc"], a["vc"], a["tbl"], a["cu"], a["sp"], scale, window, kb, ks,
                                       dtype, a["out"], a["lse"], a["ws"], ws_bytes, None,
                                       ctypes.byref(cmp.cmp_attn_dims(**d)))


def test_attention_refusals(cmp):
    assert attn(cmp, T=0) == 0 and attn(cmp, B=0, T=0) == 0
    assert cmp.lib.cmp_paged_attention(P, P, P, P, P, P, 0.1, 0, 1, 1, 1, P, P, P, 1 << 40, None, None) == 1
    assert attn(cmp, dtype=-1) == 3
    for kw in (dict(B=-1), dict(B=0), dict(T=-1), dict(Hq=7), dict(Hq=0), dict(Hk=0), dict(Hq=1032, Hk=258),
               dict(Hq=258, Hk=2, q_stride=258 * 128), dict(D=0), dict(D=40), dict(D=512), dict(q_stride=1000),
               dict(q_stride=1028), dict(page_size=8), dict(page_size=24), dict(page_size=1040), dict(block_num=0),
               dict(block_num=2 ** 27), dict(table_stride=0), dict(max_len=-1), dict(T=2 ** 29),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
               dict(window=2 ** 31), dict(kb=0), dict(ks=0), dict(kb=2 ** 31)):
        assert attn(cmp, **kw) == 2, kw
    for name in ("q", "kc", "vc", "tbl", "cu", "out", "ws"):
        assert attn(cmp, {name: None}) == 1, name
    for name in ("q", "kc", "vc", "out", "ws"):
        assert attn(cmp, {name: P + 8}) == 2, name
    for name in ("tbl", "cu", "sp", "lse"):
        assert attn(cmp, {name: P + 2}) == 2, name
    need = cmp.paged_attention_workspace(4, 8, 2, 128)
    assert need > 0 and attn(cmp, ws_bytes=need - 1) == 2


def test_attention_sequences(cmp):
    assert attn(cmp, B=2 ** 20 + 1) == 2 and attn(cmp, B=2 ** 30) == 2
    assert attn(cmp, {"q": None}, B=2 ** 20) == 1                 # the sizes are fine


def test_workspace(cmp):
    assert cmp.paged_attention_workspace(4, 8, 2, 40) == 0
    assert cmp.paged_attention_workspace(1, 8, 2, 128, 1) <= cmp.paged_attention_workspace(4096, 8, 2, 128)


def test_sizes_past_64_bits_are_refused(cmp):
    """They would wrap to small ones."""
    with pytest.raises(ValueError, match="64 bits"):
        cmp.paged_attention_workspace(2 ** 64 + 4, 8, 2, 128)
    with pytest.raises(ValueError, match="64 bits"):
        cmp.paged_attention_workspace(4, 8, 2, 128, 2 ** 64 + 1)
    assert cmp.paged_attention_workspace(2 ** 62, 8, 2, 128) == 0


def refuses_as_ever(cmp, monkeypatch):
    """The operators with their compiled binding looked for anew."""
    import torch
    for name in ("_torch", "_calls"):
        monkeypatch.setattr(cmp, name, None)
    with pytest.warns(RuntimeWarning, match="compiled binding"):
        with pytest.raises(ValueError, match="CUDA"):
            cmp.qk_norm_rope(torch.zeros(2, 4, 64, dtype=torch.bfloat16), None, torch.ones(64, dtype=torch.bfloat16))
    assert cmp._calls is None


def test_without_the_compiled_binding(cmp, monkeypatch):
    """A missing one is no reason to refuse a call: the Python one serves every call."""
    import sys
    monkeypatch.delattr(cmp, "_fast", raising=False)
    monkeypatch.setitem(sys.modules, cmp.__name__ + "._fast", None)
    refuses_as_ever(cmp, monkeypatch)


def test_compiled_binding_of_another_pytorch(cmp, monkeypatch):
    """One that was built against other headers would read tensors wrongly: it is not used."""
    import sys
    import types
    for other in (types.SimpleNamespace(torch_version="1.0.0"), types.SimpleNamespace()):
        monkeypatch.setattr(cmp, "_fast", other, raising=False)
        monkeypatch.setitem(sys.modules, cmp.__name__ + "._fast", other)
        refuses_as_ever(cmp, monkeypatch)


def test_compiled_binding_of_this_pytorch(cmp, monkeypatch):
    import torch
    for name in ("_torch", "_calls"):
        monkeypatch.setattr(cmp, name, None)
    assert cmp._torch_module() is torch and cmp._calls.torch_version == torch.__version__


def test_build_without_pytorch(monkeypatch, tmp_path):
    """The library needs no PyTorch to be built; its compiled binding is left out then, and where
    its compilation fails."""
    import importlib.util
    import os

    import streaming_kv_cache_varlen_b200 as m
    spec = importlib.util.spec_from_file_location("build_script", os.path.join(os.path.dirname(m.__file__), "_build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    with monkeypatch.context() as p:
        p.setattr(b.importlib.util, "find_spec", lambda name: None)
        assert b.build_fast(force=True) is None
    monkeypatch.setattr(b, "FAST", str(tmp_path / "fast.so"))
    monkeypatch.setattr(b, "OBJDIR", str(tmp_path))
    monkeypatch.setattr(b, "FAST_KEY", str(tmp_path / "fast.key"))
    bad = tmp_path / "bad.cpp"
    bad.write_text("#error no\n")
    monkeypatch.setattr(b, "FAST_SRC", str(bad))
    with pytest.warns(UserWarning, match="not built"):
        assert b.build_fast() is None
    ok = tmp_path / "ok.cpp"
    ok.write_text("int x;\n")
    monkeypatch.setattr(b, "FAST_SRC", str(ok))
    assert b.build_fast() == b.FAST and os.path.exists(b.FAST)
    stamp = os.stat(b.FAST).st_mtime_ns
    assert b.build_fast() == b.FAST and os.stat(b.FAST).st_mtime_ns == stamp   # up to date
    monkeypatch.setattr(b, "FAST_SRC", str(bad))
    with pytest.warns(UserWarning, match="not built"):
        assert b.build_fast(force=True) is None
    assert not os.path.exists(b.FAST)                                           # nor is the old one left
    monkeypatch.setattr(b, "FAST_SRC", str(ok))
    assert b.build_fast() == b.FAST
    stamp = os.stat(b.FAST).st_mtime_ns
    (tmp_path / "fast.key").write_text("another PyTorch")
    assert b.build_fast() == b.FAST and os.stat(b.FAST).st_mtime_ns != stamp   # built anew


def test_binding_wants_cuda_tensors(cmp):
    import torch
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    c = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        cmp.qk_norm_rope(q, None, w)
    with pytest.raises(ValueError, match="CUDA"):
        cmp.kv_append(q, q, c, c, i[None], i)
    with pytest.raises(ValueError, match="CUDA"):
        cmp.paged_attention(q, c, c, i[None], i)
    with pytest.raises(TypeError, match="Tensor"):
        cmp.paged_attention(None, c, c, i[None], i)
