"""The compiled checks of tensor arguments raise SpecError whatever torch says of a tensor: a C++
exception there ends no process.  In a process of its own, which an abort would end."""
import subprocess
import sys
import os

import pytest

pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SETUP = """
import torch
from speculative_decoding_draft_04_gb300 import _lib, build
build.build()
_lib._types()
def addresses(*a):
    try:
        _lib._args.addresses(-1, *a)
    except _lib.SpecError as e:
        print("refused:", e)
"""


def says(code):
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", SETUP + code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    return r.stdout


def test_a_nested_tensor():
    out = says("""
x = torch.nested.nested_tensor([torch.zeros(2), torch.zeros(3)])
addresses("slots", x, torch.float32, (2,))
addresses("k", x, None, (2, 2, 2))
""")
    assert out.count("refused:") == 2


def test_a_sparse_tensor():
    out = says("""
x = torch.zeros((4, 2, 64)).to_sparse()
addresses("k", x, None, (4, 2, 64))
addresses("slots", x, torch.float32, (4, 2, 64))
""")
    assert out.count("refused:") == 2


def test_a_tensor_without_storage():
    out = says("""
x = torch.zeros((4, 2, 64), device="meta")
addresses("k", x, None, (4, 2, 64))
addresses("slots", x, torch.float32, (4, 2, 64))
addresses("slots", x, torch.float32, (4, -1, 2 ** 70))
""")
    assert out.count("refused:") == 3
