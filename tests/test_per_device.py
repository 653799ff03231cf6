"""csrc/per_device.h on its own: what the host keeps belongs to a device."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exl3_trellis_quantized_rot_gb300", "csrc")


def run(tmp_path, body):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text('#include "per_device.h"\n#include <cassert>\nint main() {\n' + body + "\n}\n")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    subprocess.run([str(exe)], check=True)


def test_each_device_has_its_own_value_and_a_failure_is_not_kept(tmp_path):
    run(tmp_path, """
  tfx::PerDevice<int*> p;
  int words[3] = {}, looked = 0;
  bool works = false;
  auto find = [&](int d) { return [&looked, &works, &words, d]() -> int* { looked++; return works ? words + d : nullptr; }; };
  assert(!p.of(0, find(0)) && looked == 1);
  works = true;
  assert(p.of(0, find(0)) == words && looked == 2);
  assert(p.of(1, find(1)) == words + 1 && p.of(0, find(0)) == words && p.of(1, find(1)) == words + 1 && looked == 3);
  assert(p.of(-1, find(2)) == words + 2 && p.of(64, find(2)) == words + 2 && looked == 5);
""")


def test_a_kernel_setting_holds_on_its_device(tmp_path):
    run(tmp_path, """
  tfx::KernelSettings<3> s;
  const char k[4] = {};
  assert(!s.find(k, 0) && !s.find(nullptr, 0 + 1));
  s.note(k, 0, 5);
  assert(s.find(k, 0) && *s.find(k, 0) == 5 && !s.find(k, 1) && !s.find(k + 1, 0));
  s.note(k, 1, 6);
  s.note(k, 0, 7);  // a new value in the old one's place
  s.note(k + 1, 0, 8);
  assert(*s.find(k, 0) == 7 && *s.find(k, 1) == 6 && *s.find(k + 1, 0) == 8);
  s.note(k + 2, 0, 9);  // no room: the oldest goes, and is set again when it is next used
  assert(!s.find(k, 0) && *s.find(k, 1) == 6 && *s.find(k + 1, 0) == 8 && *s.find(k + 2, 0) == 9);
""")
