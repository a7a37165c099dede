"""Edges of the layer operators' host side: statuses, refusals, empty calls, builds."""
import ctypes

import pytest
import torch

from chunked_linear_recurrence_gated_gb300 import build, gdn

P = ctypes.c_void_p
FAKE = 1 << 20  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


def test_exchange_check_refuses_bad_arguments(lib):
    for sums, silent in ((None, -1), (FAKE + 2, -1), (FAKE, -2), (FAKE, 4)):
        assert lib.gdn_diag_exchange(P(sums) if sums else None, silent, 20, None) == 1


def test_rows_of_empty_tensors(lib):
    """Any layout of no rows is one stride; what has rows is checked as before."""
    e, z = torch.empty, torch.zeros
    assert gdn._rows("q", e(2, 0, 3, 64), 2) == 192
    assert gdn._rows("q", e(0, 5, 3, 64), 2) == 192
    assert gdn._rows("g", e(3, 0, 4), 1) == 4
    assert gdn._rows("q", z(4, 8, 16)[:2, :0, 8:], 1) == 8
    with pytest.raises(ValueError):
        gdn._rows("q", z(4, 8, 16)[:2, :1, ::2], 1)
    with pytest.raises(ValueError):
        gdn._rows("q", z(4, 8, 16)[:2, :3], 1)


# ------------------------------------------------------------------------------ build
@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """build() into an empty folder, of one small kernel file."""
    monkeypatch.setattr(build, "OUT", str(tmp_path))
    for name, file in (("LIB", "libgdn.so"), ("EXT", "_gdn_torch.so"), ("EXT_FOR", "_gdn_torch.for")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    one = [s for s in build.sources() if s.endswith("gdn_noalloc.cu")]
    monkeypatch.setattr(build, "sources", lambda: one)
    return tmp_path


def test_the_library_builds_without_torch(elsewhere, monkeypatch):
    found = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else found(name, *a))
    assert build.build() == str(elsewhere / "libgdn.so")
    assert (elsewhere / "libgdn.so").exists() and not (elsewhere / "_gdn_torch.so").exists()
    made = (elsewhere / "libgdn.so").stat().st_mtime_ns
    build.build()
    assert (elsewhere / "libgdn.so").stat().st_mtime_ns == made


def test_the_library_is_linked_when_the_python_entry_does_not_compile(elsewhere, monkeypatch):
    bad = elsewhere / "bad.cpp"
    bad.write_text("this is not C++\n")
    monkeypatch.setattr(build, "EXT_SRC", str(bad))
    with pytest.raises(RuntimeError, match="bad.cpp"):
        build.build()
    assert (elsewhere / "libgdn.so").exists() and not (elsewhere / "_gdn_torch.so").exists()


def test_a_module_of_another_torch_is_not_loaded(lib, tmp_path, monkeypatch):
    """The module is compiled against torch's headers: another version's tensors have
    another layout."""
    other = tmp_path / "for"
    other.write_text("3.12\n__version__ = '2.0.0'\n")
    monkeypatch.setattr(build, "EXT_FOR", str(other))
    monkeypatch.setattr(gdn, "_ext_module", None)
    with pytest.raises(RuntimeError, match="another torch"):
        gdn.ext()
