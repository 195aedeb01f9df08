"""What the build step compiles and when, on the host alone: the C library
needs no PyTorch headers, and an extension module that was built against
another PyTorch is neither taken for current nor loaded."""
import importlib.util
import os
import sys

import pytest

from serving_moe_route_gb300 import _build, decode


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the build step with small sources of its own."""
    pkg = tmp_path / "pkg"
    (pkg / "csrc").mkdir(parents=True)
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "moe_route.h").write_text("int moe_one(void);\n")
    (pkg / "csrc" / "one.cu").write_text('extern "C" int moe_one() { return 1; }\n')
    (pkg / "csrc" / "decode_ext.cpp").write_text("#error no headers here\n")
    (pkg / "_build.py").write_text(open(_build.__file__).read())
    spec = importlib.util.spec_from_file_location("build_copy", pkg / "_build.py")
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_library_needs_no_headers_of_pytorch(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # an import of it fails
    assert tree.build(extension=False) == tree.LIB_PATH
    assert os.path.exists(tree.LIB_PATH) and not os.path.exists(tree.EXT_PATH)
    assert tree.up_to_date()


def test_an_extension_that_does_not_compile_leaves_the_library(tree):
    with pytest.raises(RuntimeError, match="decode_ext.cpp"):
        tree.build()
    assert tree.up_to_date() and not tree.ext_up_to_date()
    before = os.path.getmtime(tree.LIB_PATH)
    with pytest.raises(RuntimeError, match="decode_ext.cpp"):
        tree.build()  # tried again, the library is not
    assert os.path.getmtime(tree.LIB_PATH) == before


def test_an_extension_of_another_pytorch_is_built_anew(tree, monkeypatch):
    with open(tree.EXT_SRC, "w") as f:
        f.write("int moe_nothing() { return 0; }\n")
    tree.build()
    assert tree.ext_up_to_date()
    first = os.path.getmtime(tree.EXT_PATH)
    tree.build()
    assert os.path.getmtime(tree.EXT_PATH) == first
    import torch

    monkeypatch.setattr(torch, "__version__", "1.0.other")
    assert tree.up_to_date() and not tree.ext_up_to_date()
    tree.build()
    assert tree.ext_up_to_date() and os.path.getmtime(tree.EXT_PATH) > first


def test_an_extension_of_another_pytorch_is_not_loaded(monkeypatch, tmp_path):
    fake = tmp_path / "moe_decode_ext.so"
    fake.write_bytes(b"never read")
    monkeypatch.setattr(decode, "_ext_module", None)
    monkeypatch.setattr(_build, "EXT_PATH", str(fake))
    monkeypatch.setattr(_build, "EXT_STAMP", str(fake) + ".torch")
    for stamp in (None, "torch 1.0.other cxx11 1\n"):
        if stamp:
            (tmp_path / "moe_decode_ext.so.torch").write_text(stamp)
        with pytest.raises(RuntimeError, match="another PyTorch"):
            decode._ext()
