"""No C++ exception leaves the token operators' C entries."""

from __future__ import annotations

import ctypes
import os
import re
import shutil
import subprocess

import pytest

import lidar_point_cloud_gb300 as pv
from lidar_point_cloud_gb300 import _build
from test_tokens_abi import lib  # noqa: F401

THROWER = r"""
#include <new>
#include <system_error>
namespace pvs { int caught() noexcept; }
extern "C" int thrown(int which) try {
  if (which == 0) throw std::bad_alloc();
  if (which == 1) throw std::system_error(std::make_error_code(std::errc::resource_deadlock_would_occur));
  throw which;
} catch (...) {
  return pvs::caught();
}
"""


@pytest.mark.parametrize("source", ["pv_rope.cu", "pv_scan.cu", "pv_attn.cu"])
def test_every_entry_ends_in_a_handler(source):
    with open(os.path.join(_build.CSRC, source)) as f:
        text = f.read()
    entries = re.findall(r'^extern "C" int pv_\w+\(.*?^}$', text, re.M | re.S)
    assert entries
    for entry in entries:
        assert re.search(r"\) try \{\n", entry) and "\n} catch (...) {\n  return caught();\n}" in entry, entry.splitlines()[0]


def test_what_the_handler_answers(lib, tmp_path):  # noqa: F811
    if not shutil.which("g++"):
        pytest.skip("no g++")
    source, out = tmp_path / "thrower.cpp", tmp_path / "thrower.so"
    source.write_text(THROWER)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", str(source), "-o", str(out), pv._binding.lib_path(),
                    f"-Wl,-rpath,{os.path.dirname(pv._binding.lib_path())}"], check=True)
    thrown = ctypes.CDLL(str(out)).thrown
    assert [thrown(n) for n in range(3)] == [-3, -4, -4]
