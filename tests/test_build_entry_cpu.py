"""The build entry point on a tree that was never built: it compiles first and imports the package
after that.  (nvcc is stood in for by a script that hands out the library built here.)"""

import os
import shutil
import stat
import subprocess
import sys

from tests._sana import ROOT, _lib


def test_build_on_a_fresh_checkout(tmp_path):
    tree = tmp_path / "tree"
    pkg = "softmax_attention_sana_b200"
    tree.mkdir()
    shutil.copy(os.path.join(ROOT, "__graft_entry__.py"), tree)
    shutil.copytree(os.path.join(ROOT, "include"), tree / "include")
    shutil.copytree(os.path.join(ROOT, pkg), tree / pkg,
                    ignore=shutil.ignore_patterns("*.so", "_build", "__pycache__"))
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(f"""#!{sys.executable}
import shutil, sys
out = sys.argv[sys.argv.index("-o") + 1]
shutil.copy({_lib.LIB_PATH!r}, out) if "-shared" in sys.argv else open(out, "w").close()
""")
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    (tree / "tests").mkdir()
    shutil.copy(os.path.join(ROOT, "tests", "_sana.py"), tree / "tests")
    lib = tree / pkg / "libsana.so"
    for code in ("import __graft_entry__ as g; g.build(); import softmax_attention_sana_b200 as s; print(s.__file__)",
                 "from tests._sana import sana; print(sana.__file__)"):
        run = subprocess.run([sys.executable, "-c", code], cwd=tree, capture_output=True, text=True, timeout=300,
                             env={**os.environ, "NVCC": str(nvcc), "PYTHONPATH": ""})
        assert run.returncode == 0, run.stderr
        assert run.stdout.startswith(str(tree)) and lib.exists()
        lib.unlink()
