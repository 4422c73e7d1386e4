"""The package without torch or without what is built: it imports, and calls say what is missing."""
import os
import subprocess
import sys

import memory_bound_elementwise_gb300 as ew

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    return r.stdout


def test_star_import_without_torch():
    out = run("import sys; sys.modules['torch'] = None\n"
              "from memory_bound_elementwise_gb300 import *\n"
              "assert callable(ew_add) and callable(lib)\n"
              "try:\n    ew_embed(None, None)\n"
              "except ImportError as e:\n    print('refused:', e)\n")
    assert out.startswith("refused:") and "torch" in out


def test_star_import_without_the_library():
    out = run("import memory_bound_elementwise_gb300 as ew\n"
              "ew.LIB_PATH = '/nonexistent/libew.so'\n"
              "from memory_bound_elementwise_gb300 import *\n"
              "for call in (lambda: lib(), lambda: ew_embed(None, None)):\n"
              "    try:\n        call()\n"
              "    except RuntimeError as e:\n        print('refused:', e)\n")
    assert out.count("refused: libew.so is not built") == 2


def test_every_public_name_is_there():
    out = run("from memory_bound_elementwise_gb300 import *\n"
              "import memory_bound_elementwise_gb300 as ew\n"
              "assert all(n in globals() for n in ew.__all__)\n"
              "print(len(ew.__all__))\n")
    assert int(out) == len(ew.__all__) and "ew_embed" in ew.__all__
