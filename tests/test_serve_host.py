"""Host side of the paged serving operators (no GPU): pins of the oracle, what the C
entries refuse and accept without touching a device."""

import ctypes
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest

from oracle import serve_oracle as S


def test_slots_oracle_gives_unserved_requests_no_length():
    # request 1 wants two pages of one; request 2 none; request 3 is out of range
    got = S.slots([0, 0, 3, -2], [4, 5, 1, 3], np.zeros((4, 2), int), [0, 0, 1, 0],
                  np.array([4, 5]), 2, 4, 20)
    assert got["errors"] == {"blocks", "len"} and got["held"] == [1, 0, 1, 0]
    assert got["seq_lens"] == [4, -1, 4, -1]


# ---------------------------------------------------------------- refusals

P = 1 << 20  # aligned addresses a megabyte apart, never dereferenced
ERR_ARG = -1


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_16_gb300 import build
    build.build()
    from speculative_decoding_verification_16_gb300 import binding
    return binding._lib


SLOTS = dict(ctx=P, new=2 * P, B=4, page=16, table=3 * P, stride=8, width=8, held=4 * P,
             free=5 * P, cap=64, count=6 * P, rows=10, offs=7 * P, seq=8 * P, pos=9 * P,
             slots=10 * P, held_out=11 * P, count_out=12 * P, err=13 * P, stream=None)


@pytest.mark.parametrize("result", ["offs", "seq", "pos", "slots", "held_out", "count_out"])
@pytest.mark.parametrize("read", ["ctx", "new", "held", "count"])
def test_slots_refuses_results_over_what_it_reads(lib, result, read):
    """CTAs read the lengths and counts while others write the results."""
    for shift in (0, 8 if result == "slots" else 4):  # the same place, and one in part
        last = dict(offs=16, seq=12, pos=36, slots=72, held_out=12, count_out=0)[result]
        a = {**SLOTS, result: SLOTS[read] - (last if shift else 0)}
        assert lib.spec_verify_slots(*a.values()) == ERR_ARG


def test_attention_without_rows_needs_no_rows_memory(lib):
    """An empty tensor has no address: a step without new tokens is no error."""
    ok = lib.spec_verify_attention(None, 1024, 128, P, P, 16384, 1024, 128, P, 8, 8, P, P, 4, 0, 4,
                                   8, 8, 128, 9, 16, 0, ctypes.c_float(0.1), 0, None, 1024, 128,
                                   None, None, P, 1 << 40, None)
    assert ok == 0


# ---------------------------------------------------------------- the host module

PACKAGE = "speculative_decoding_verification_16_gb300"
USE = f"""
import torch
from {PACKAGE} import binding
assert binding.spec_verify_workspace_size(32, 512) > 0
t = torch.zeros(1, 1, 8)
try:
    binding.spec_verify_append(t, t, torch.zeros(1, dtype=torch.int64), t[None], t[None])
except ImportError as e:
    print("ImportError:", e)
except ValueError as e:
    print("ValueError:", e)
"""


def use_copy(lib, tmp_path, calls, stamp):
    """The package with the built library, and the host module or not."""
    from speculative_decoding_verification_16_gb300 import build
    to = tmp_path / PACKAGE
    to.mkdir()
    for f in os.listdir(build.HERE):
        if f.endswith(".py"):
            shutil.copy(os.path.join(build.HERE, f), to)
    shutil.copy(build.LIB, to)
    if calls:
        shutil.copy(build.CALLS, to)
    if stamp is not None:
        (to / os.path.basename(build.CALLS_STAMP)).write_text(stamp)
    r = subprocess.run([sys.executable, "-c", USE], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_the_verify_step_needs_no_host_module(lib, tmp_path):
    """The library alone is enough to import the binding; a serving operator says
    what is missing."""
    out = use_copy(lib, tmp_path, False, None)
    assert out.startswith("ImportError") and "_serve_calls" in out


def test_a_host_module_of_another_torch_is_not_loaded(lib, tmp_path):
    out = use_copy(lib, tmp_path, True, "torch 1.0, cpython-30")
    assert out.startswith("ImportError") and "torch 1.0" in out


def test_the_host_module_is_loaded(lib, tmp_path):
    from speculative_decoding_verification_16_gb300 import build
    assert "CUDA device" in use_copy(lib, tmp_path, True, build.calls_stamp())


def test_build_without_a_host_compiler_keeps_the_library(lib, tmp_path, monkeypatch):
    from speculative_decoding_verification_16_gb300 import build
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_serve_calls.so"))
    monkeypatch.setattr(build, "CALLS_STAMP", str(tmp_path / "_serve_calls.so.stamp"))

    def no_compiler(tool, cmd, verbose):
        raise FileNotFoundError(tool)
    monkeypatch.setattr(build, "_run", no_compiler)
    with pytest.warns(UserWarning, match="not built"):
        assert build.build() == build.LIB


def test_build_renews_the_host_module_for_another_torch(lib, tmp_path, monkeypatch):
    from speculative_decoding_verification_16_gb300 import build
    assert build.calls_built_for() == build.calls_stamp()
    monkeypatch.setattr(build, "CALLS_STAMP", str(tmp_path / "stamp"))
    (tmp_path / "stamp").write_text("torch 1.0, cpython-30")
    built = []
    monkeypatch.setattr(build, "_build_calls", built.append)
    build.build()
    assert built == [False]
