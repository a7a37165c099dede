"""Edges of the layer operators' host side: statuses, refusals, empty calls, builds."""
import ctypes

import numpy as np
import pytest
import torch

import step_precision as sp
from chunked_linear_recurrence_gated_gb300 import build, gdn
from oracle import layer_ops as lo

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


# -------------------------------------------------- the bound of the step's GPU tests
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_the_step_bound_tells_two_tf32_parts_from_one(bf16, dk, dv):
    """The tile algorithm with operands in two TF32 parts stays far inside the bound of
    the GPU tests; with one part per operand every head of every length is outside."""
    rng = np.random.default_rng(dk + bf16)
    f32 = lambda *s: rng.standard_normal(s).astype(np.float32)
    kept = lambda x: torch.from_numpy(x).bfloat16().float().numpy() if bf16 else x
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)
    for T in (2, 3, 8, 9, 16, 33):
        q, k = kept(unit(f32(T, 2, dk))), kept(unit(f32(T, 2, dk)))
        v, S = kept(f32(T, 2, dv)), 0.1 * f32(1, 2, dk, dv)
        g, beta = kept(-lo.softplus(f32(T, 2))), kept(lo.sigmoid(f32(T, 2)))
        args = (q, k, v, g, beta)
        ro, rS = lo.step(*[x.astype(np.float64) for x in (*args, S)], cu=[0, T])
        for h in range(2):
            a = [np.ascontiguousarray(x[:, h]) for x in args]
            for parts in (1, 2):
                o, S1 = sp.tiles(*a, S[0, h], parts, bf16)
                errs = [sp.error(S1[None], rS[0, h][None])]
                if not bf16:
                    errs.append(sp.error(o[None], ro[:, h][None]))
                if parts == 2:
                    assert max(errs) <= 0.1 * sp.bound([T]), (T, h, errs)
                else:
                    assert min(errs) > 2.0 * sp.bound([T]), (T, h, errs)


# ------------------------------------------------------------------ the end of int
def refused(status):
    """The status of a call whose sizes are refused on the host. (Without that check it
    would try to launch, which fails here where there is no GPU.)"""
    return status == 2


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 2 ** 14])
def test_sizes_whose_row_indices_would_wrap_are_refused(lib, rows):
    """A thread's next rows, sequences and channels are 32-bit numbers a few thousand
    past its present ones."""
    at = lambda n, ws=None: [P(FAKE)] * n + ([P(FAKE), 1 << 40] if ws else []) + [None]
    s = gdn.gdn_res_norm_shape(rows, 8, 1, 1, 1e-6)
    assert lib.gdn_res_norm_workspace_bytes(s) == 0
    assert refused(lib.gdn_res_norm_fwd(s, *at(7)))
    assert refused(lib.gdn_res_norm_bwd(s, *at(12, True)))
    conv = lambda N, C: gdn.gdn_conv_step_shape(N, 0, N, C, 4, 1, 1, C)
    assert refused(lib.gdn_conv_step(conv(rows, 64), *at(9)))
    assert refused(lib.gdn_conv_step(conv(1, rows // 4 * 4), *at(9)))
    assert not refused(lib.gdn_conv_step(conv(0, 64), *at(9)))
