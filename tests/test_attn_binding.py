"""The host side of the attention binding and the arithmetic of its work list, without a GPU."""
import os
import random
import subprocess

import pytest
import torch

from int4_routed_expert_quantize_gb300 import _build, attn


def test_page_table_rows_are_where_the_tensor_has_them():
    """an expanded row has stride 0 and holds no second row behind it; rows that overlap are refused"""
    flat = torch.arange(40, dtype=torch.int32)
    assert attn._row_stride(flat.view(4, 10)) == 10
    assert attn._row_stride(flat.view(4, 10)[:, :7]) == 10
    assert attn._row_stride(flat.view(4, 10)[:1]) == 10
    assert attn._row_stride(flat[None, :5].expand(3, -1)) == 0
    assert attn._row_stride(torch.as_strided(flat, (1, 10), (3, 1))) == 10
    for rows, width, stride in ((3, 10, 4), (2, 2, 1)):
        with pytest.raises(ValueError):
            attn._row_stride(torch.as_strided(flat, (rows, width), (stride, 1)))


def host_program(tmp_path, body):
    """a program over csrc/attn_stretch.h that ends with an error at undefined operations; -> a call of it on lines"""
    src, exe = tmp_path / "stretch.cpp", str(tmp_path / "stretch")
    src.write_text('#include <cstdio>\n#include "attn_stretch.h"\nusing namespace coli;\nint main() {\n' + body + "}\n")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", _build.CSRC,
                           str(src), "-o", exe])

    def call(rows):
        text = "".join(" ".join(map(str, r)) + "\n" for r in rows)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
        assert out.returncode == 0, out.stderr[-500:]
        return [int(x) for x in out.stdout.split()]
    return call


def test_stretches_of_long_lists(tmp_path):
    """the smallest length that covers the list with the CTAs and whose square reaches a twelfth of the longest unit"""
    call = host_program(tmp_path, """
  unsigned run, ctas;
  int longest;
  while (scanf("%u %u %d", &run, &ctas, &longest) == 3) printf("%u\\n", list_stretch(run, ctas, longest));
  return 0;
""")
    r = random.Random(0)
    rows = [(0, 304, 0), (1, 304, 1), (110, 304, 110), (13378 * 304, 304, 15000), (14000 * 304, 304, 16384),
            (2 ** 31 - 1, 304, 2 ** 24), (2 ** 31 - 1, 1, 2 ** 24), (46341 * 152, 152, 5), (65536 * 304, 304, 2 ** 24)]
    rows += [(int(2 ** r.uniform(0, 31)), r.choice([152, 304]), int(2 ** r.uniform(0, 24))) for _ in range(500)]
    for (run, ctas, longest), per in zip(rows, call(rows)):
        want = max(1, -(-run // ctas))
        while want * want * 12 < longest:
            want += 1
        assert per == want, (run, ctas, longest)


def test_lengths_of_lists_stop_when_full(tmp_path):
    call = host_program(tmp_path, """
  unsigned a, b;
  while (scanf("%u %u", &a, &b) == 2) printf("%u\\n", list_add(a, b));
  return 0;
""")
    full = 2 ** 31 - 1
    r = random.Random(1)
    rows = [(0, 0), (full, full), (full, 0), (0, full), (full - 1, 1), (full - 1, 0), (2 ** 30, 2 ** 30), (2 ** 30, 2 ** 30 - 1)]
    rows += [(min(full, int(2 ** r.uniform(0, 31))), min(full, int(2 ** r.uniform(0, 31)))) for _ in range(500)]
    assert call(rows) == [min(full, a + b) for a, b in rows]


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """the build's commands, recorded instead of run, its outputs in a scratch folder"""
    seen = []
    monkeypatch.setattr(_build.subprocess, "check_call", lambda cmd, **kw: seen.append(cmd))
    for name in ("SO", "PY_SO", "PY_TAG"):
        monkeypatch.setattr(_build, name, str(tmp_path / os.path.basename(getattr(_build, name))))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path))
    return seen


def test_the_c_library_is_built_whatever_becomes_of_the_python_side(commands, monkeypatch):
    def broken(verbose=False):
        raise subprocess.CalledProcessError(1, "attn_py.cpp")
    monkeypatch.setattr(_build, "compile_py", broken)
    with pytest.raises(subprocess.CalledProcessError):
        _build.build()
    assert any("-shared" in c and _build.SO in c for c in commands)
    assert not os.path.exists(_build.PY_TAG)


def test_without_torch_the_c_library_alone_is_built(commands, monkeypatch):
    monkeypatch.setattr(_build, "torch_tag", lambda: None)
    _build.build()
    assert any("-shared" in c and _build.SO in c for c in commands)
    assert not any("attn_py" in str(c) for c in commands)


def test_no_fixed_place_of_cuda(commands):
    _build.build()
    assert any("attn_py" in str(c) for c in commands) and not any("/usr/local/cuda" in str(c) for c in commands)


def test_another_torch_makes_the_build_stale(commands, monkeypatch):
    _build.build()
    for p in (_build.SO, _build.PY_SO):
        open(p, "w").close()
    assert not _build.is_stale()
    monkeypatch.setattr(_build, "torch_tag", lambda: "torch 0.0, cpython-312")
    assert _build.is_stale()
