"""Programs that link libew.so, and the binding that does."""
import os
import shutil
import subprocess
import sys

import pytest

import memory_bound_elementwise_gb300 as ew

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(not os.path.exists(ew.LIB_PATH), reason="libew.so not built")


def test_a_client_linked_by_path_finds_the_library(tmp_path):
    """Without a run path: the client names the file that it was linked with."""
    cc = shutil.which("cc") or shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    source, out = tmp_path / "client.c", tmp_path / "client"
    source.write_text('#include <stdio.h>\n#include "ew.h"\nint main(void) { printf("%d", ew_version()); return 0; }\n')
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(source), ew.LIB_PATH, "-o", str(out)], check=True)
    env = {k: v for k, v in os.environ.items() if k != "LD_LIBRARY_PATH"}
    r = subprocess.run([str(out)], cwd="/", env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0 and int(r.stdout) == ew.lib().ew_version(), r.stdout


def test_the_binding_uses_the_same_library(tmp_path):
    """One copy in a process, wherever the package lies: its settings hold for both ways in."""
    moved = tmp_path / "memory_bound_elementwise_gb300"
    here = os.path.dirname(os.path.abspath(ew.__file__))
    os.makedirs(moved / "_lib")
    for name in os.listdir(here):
        if name.endswith(".py"):
            shutil.copy(os.path.join(here, name), moved / name)
    for name in ("libew.so", "_ew_torch.so"):
        if not os.path.exists(os.path.join(here, "_lib", name)):
            pytest.skip(name + " not built")
        shutil.copy(os.path.join(here, "_lib", name), moved / "_lib" / name)
    code = ("import memory_bound_elementwise_gb300 as ew\new.ew_embed\n"
            "print(sorted({l.split()[-1] for l in open('/proc/self/maps') if 'libew.so' in l}))")
    r = subprocess.run([sys.executable, "-c", code], cwd=str(tmp_path), stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0 and r.stdout.strip() == str([str(moved / "_lib" / "libew.so")]), r.stdout
