"""Test helper: build libsana.so if needed and import the binding."""
import os
import runpy
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

# by path: the package itself cannot be imported before its library is there
runpy.run_path(os.path.join(ROOT, "softmax_attention_sana_b200", "build.py"))["build"]()

import softmax_attention_sana_b200 as sana  # noqa: E402,F401
from softmax_attention_sana_b200 import _lib  # noqa: E402,F401
