"""The binding without its compiled module, and its build without a compiler for it (no GPU)."""
import os
import warnings

import pytest

import test_binding
from sliding_window_attention_router_gb300 import build


@pytest.fixture(scope="module")
def swa():
    build.build()
    import sliding_window_attention_router_gb300 as m
    return m


def test_the_compiled_calls_are_used_where_they_were_built(swa, monkeypatch):
    monkeypatch.setattr(swa, "_compiled", None)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert swa._calls().__name__.endswith("._binding")


@pytest.mark.parametrize("stamp", [None, "PyTorch 1.0.0, Python 3.12"])
def test_another_pytorch_takes_the_python_calls(swa, monkeypatch, tmp_path, stamp):
    path = tmp_path / "torch_version"
    if stamp:
        path.write_text(stamp)
    monkeypatch.setattr(swa, "_compiled", None)
    monkeypatch.setattr(build, "TORCH", str(path))
    with pytest.warns(RuntimeWarning, match="another PyTorch"):
        calls = swa._calls()
    assert calls.__name__.endswith("._python_calls") and swa._calls() is calls
    test_binding.test_calls_refuse_host_tensors_and_other_objects(swa)
    test_binding.test_axes_are_small_whole_numbers(swa)


def test_both_take_the_same_arguments(swa):
    """Every call of the compiled module is there in Python, with as many arguments."""
    import inspect

    from sliding_window_attention_router_gb300 import _binding, _python_calls
    for name in ("rope", "append_paged", "decode_tree", "accept_tree", "fork_paged"):
        n = len(inspect.signature(getattr(_python_calls, name)).parameters)
        with pytest.raises(ValueError, match=f"{n + 1} arguments, expected {n}$"):
            getattr(_binding, name)(*[None] * (n + 1))


@pytest.mark.parametrize("why", [RuntimeError("g++ failed on binding.cpp"), FileNotFoundError("g++")])
def test_a_failed_binding_leaves_the_library_built(swa, monkeypatch, tmp_path, why):
    """The library is built (or found fresh) whatever becomes of the binding, which is tried again."""
    tries = []

    def fail():
        tries.append(0)
        raise why

    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "_build_binding", fail)
    before = os.path.getmtime(build.LIB)
    for n in (1, 2):
        with pytest.warns(RuntimeWarning, match="not built: g"):
            assert build.build() == build.LIB
        assert len(tries) == n and os.path.getmtime(build.LIB) == before


def test_a_failed_compiler_leaves_no_old_binding_in_use(monkeypatch, tmp_path):
    """An object of an older header must not be bound to a newer library."""
    stamp = tmp_path / "torch_version"
    stamp.write_text(build._against())
    monkeypatch.setattr(build, "TORCH", str(stamp))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    assert build.same_torch()
    monkeypatch.setattr(build, "_BINDING_SOURCE", "no_such_source.cpp")
    with pytest.raises(RuntimeError, match="failed"):
        build._build_binding()
    assert not build.same_torch()
