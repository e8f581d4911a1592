"""When the torch side of the package is built: beside the library, for the installed torch and Python,
and not at all where there is no torch. No compiler runs here."""
import importlib.util
import os
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(monkeypatch, tmp_path):
    """_build.py on files of its own; `ran` lists the compilers' output files."""
    spec = importlib.util.spec_from_file_location("gqa_build_test", os.path.join(ROOT, "grouped_query_softmax_b200", "_build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.LIB, m.CALLS = str(tmp_path / "libgqa.so"), str(tmp_path / "_torch_calls.so")
    m.ran = []

    def compiler(cmd):
        out = cmd[cmd.index("-o") + 1]
        m.ran.append(os.path.basename(out).split(".so")[0])
        with open(out, "wb") as f:
            f.write(b"\0".join(c.encode() for c in cmd).replace(b'"', b"\0"))

    monkeypatch.setattr(m, "subprocess", types.SimpleNamespace(check_call=compiler))
    torch = tmp_path / "torch"
    (torch / "lib").mkdir(parents=True)
    (torch / "lib" / "libc10_cuda.so").touch()
    (torch / "version.py").write_text("__version__ = '9.1.0+cu999'\n")
    m.torch, real = torch, importlib.util.find_spec
    m.found = types.SimpleNamespace(submodule_search_locations=[str(torch)])
    monkeypatch.setattr(m.importlib.util, "find_spec", lambda name: m.found if name == "torch" else real(name))
    return m


def test_both_files_are_built_once(build):
    assert build.stale()
    build.build()
    assert build.ran == ["libgqa", "_torch_calls"] and not build.stale()
    build.build()
    assert build.ran == ["libgqa", "_torch_calls"]
    build.build(force=True)
    assert build.ran == ["libgqa", "_torch_calls"] * 2


@pytest.mark.parametrize("what", ["no torch", "no CUDA"])
def test_the_library_is_built_without_torch(build, what, capsys):
    if what == "no torch":
        build.found = None
    else:
        (build.torch / "lib" / "libc10_cuda.so").unlink()
    assert build.stale()
    assert build.build() == build.LIB and build.build(force=True) == build.LIB
    assert build.ran == ["libgqa", "libgqa"] and not build.stale() and "_torch_calls.so" in capsys.readouterr().out


def test_another_torch_or_python_means_a_new_module(build, monkeypatch):
    build.build()
    build.ran.clear()
    (build.torch / "version.py").write_text("__version__ = '9.1.0+cu9999'\n")
    build.build()
    assert build.ran == ["_torch_calls"] and not build.stale()
    monkeypatch.setattr(build, "sysconfig", types.SimpleNamespace(get_config_var=lambda n: "cpython-399",
                                                                  get_paths=build.sysconfig.get_paths))
    build.build()
    assert build.ran == ["_torch_calls"] * 2 and not build.stale()


def test_the_built_module_names_its_versions():
    torch = pytest.importorskip("torch")
    import grouped_query_softmax_b200 as gqa
    doc = (gqa._calls or gqa._load_calls()).__doc__
    assert torch.__version__ in doc and doc.startswith("built for torch")
