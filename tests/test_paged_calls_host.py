"""The compiled calls of the paged cache (``csrc/paged_call.c``) are an addition: without
them the library builds, and the calls go through Python's own checks."""

import ctypes
import os
import sysconfig

import pytest

torch = pytest.importorskip("torch")

from exact_attention_15_gb300 import binding, build, paged  # noqa: E402


def _no_headers(monkeypatch, tmp_path):
    """A build whose Python has no headers, with a compiled module of an older source."""
    calls = tmp_path / os.path.basename(build.CALLS_LIB)
    monkeypatch.setattr(build, "CALLS_LIB", str(calls))
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    calls.write_bytes(b"")
    os.utime(calls, (0, 0))
    return calls


@pytest.mark.parametrize("compiler", [True, False])
def test_library_builds_without_python_headers_or_a_c_compiler(monkeypatch, tmp_path, capfd, compiler):
    build.build()
    calls = _no_headers(monkeypatch, tmp_path)
    if not compiler:
        def missing(cmd, **kw):
            raise FileNotFoundError(cmd[0])
        monkeypatch.setattr(build.subprocess, "run", missing)
    assert build.build() == build.LIB  # (the library itself is there and new)
    assert not calls.exists()
    assert "paged_call.c was not built" in capfd.readouterr().err


def test_compiled_calls_are_built_where_they_can_be():
    build.build()
    assert os.path.exists(build.CALLS_LIB)
    paged._load_calls()


def test_a_module_for_another_python_is_not_loaded(monkeypatch, tmp_path):
    """Its name carries the interpreter's tag, so that one left by another version is neither
    found fresh nor loaded."""
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert suffix != ".so" and build.CALLS_LIB.endswith(suffix)
    for name in ("_paged_call.so", "_paged_call.cpython-39-other.so"):
        (tmp_path / name).write_bytes(b"not this interpreter's")
    monkeypatch.setattr(paged, "_calls", None)
    monkeypatch.setattr(paged, "library_path", lambda: str(tmp_path / "libattn_gb300.so"))
    assert paged._load_calls() is paged._PythonCalls


def test_calls_go_through_python_without_the_module(monkeypatch, tmp_path):
    build.build()
    monkeypatch.setattr(paged, "_calls", None)
    monkeypatch.setattr(paged, "library_path", lambda: str(tmp_path / "libattn_gb300.so"))
    calls = paged._load_calls()
    for f in (calls.append, calls.decode, calls.forward):
        assert f(0, -1, None) is NotImplemented

    # host tensors stand in for those of a device with the index -1; no call here may pass the
    # checks of its arguments
    struct = paged._PagedCacheStruct(k=0x10000, v=0x10000, num_pages=4, page_size=16, H_kv=2, d=64, type=0,
                                     k_page_stride=2048, v_page_stride=2048)

    class HostCache:
        device, d, H_kv, page_size, num_pages = torch.device("cpu"), 64, 2, 16, 4
        _index, _decode_bytes, _lib = -1, 256, binding.load()
        _ref, _calls = ctypes.addressof(struct), calls

    c, i32 = HostCache(), torch.int32
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    q, k, lens, table, cu = t(3, 4, 64), t(3, 2, 64), t(3, dtype=i32), t(3, 5, dtype=i32), t(4, dtype=i32)
    for match, call in (
            ("kv_lens", lambda: binding.paged_decode(c, q, table, lens.long())),
            ("page_table", lambda: binding.paged_decode(c, q, table[:2], lens)),
            ("not a multiple", lambda: binding.paged_decode(c, t(3, 3, 64), table, lens)),
            ("cu_seqlens is required", lambda: binding.paged_forward(c, q, table, lens, None)),
            ("cu_seqlens must be", lambda: binding.paged_forward(c, q, table, lens, cu[:3])),
            ("v must be", lambda: binding.paged_append(c, q, k, t(2, 2, 64), table, lens)),
            ("q_out without q", lambda: binding.paged_append(c, None, k, k, table, lens, q_out=q))):
        with pytest.raises(ValueError, match=match):
            call()
