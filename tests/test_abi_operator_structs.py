"""The parameter structs of the tree attention, path commit, attention-weight totals and eviction have
the C compiler's size and field offsets."""
import ctypes
import os
import shutil
import subprocess

import pytest

from compressed_decode_attention_zkv_b200 import zkv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"zkv_tree_params": zkv.TreeParams, "zkv_tree_commit_params": zkv.TreeCommitParams,
           "zkv_weights_params": zkv.WeightsParams, "zkv_evict_params": zkv.EvictParams}


def test_layout(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "zkv.h"', "int main(void) {"]
    want = []
    for name, cls in STRUCTS.items():
        lines.append(f'  printf("%zu\\n", sizeof({name}));')
        want.append((name, ctypes.sizeof(cls)))
        for f, _ in cls._fields_:
            lines.append(f'  printf("%zu\\n", offsetof({name}, {f}));')
            want.append((f"{name}.{f}", getattr(cls, f).offset))
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [(n, int(x)) for (n, _), x in zip(want, got)] == want
