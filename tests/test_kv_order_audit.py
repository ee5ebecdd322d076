"""CPU audit of how the kernels over the paged cache find their rows (no GPU): tests/kv_order_audit.hip enumerates the
searches, slots, blocks and rows of csrc/kv_index.hpp over starts that rise and that do not; planted mistakes (in a copy)
make it fail."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_precision_row_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


def _run(tmp_path, include):
    exe = str(tmp_path / "kv_order_audit")
    b = subprocess.run([HIPCC, "-std=c++17", "-O1", "-x", "hip", "--cuda-host-only", "-I" + include, "-I" + CSRC,
                        os.path.join(ROOT, "tests", "kv_order_audit.hip"), "-o", exe], capture_output=True, text=True)
    assert b.returncode == 0, b.stdout + b.stderr
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


def test_every_row_is_in_bounds(tmp_path):
    r = _run(tmp_path, CSRC)
    assert r.returncode == 0 and r.stdout.startswith("ok:"), r.stdout[-1000:]


@pytest.mark.parametrize("old,new,what", [
    ("if (j < 0) return none;", "", "tokens outside the page"),
    ("if (r0 < 0) return -1;", "", "a block outside its sequence"),
    ("return lo;\n  }\n}", "return lo + 1;\n  }\n}", "sequence"),
    ("i >= n || i >= max_q_len ? -1 : i", "i >= max_q_len ? -1 : i", "a token outside"),
    ("return all <= small || r0 >= all || r0 / group", "return all <= small || r0 / group", "a block outside its sequence"),
])
def test_planted_mistakes_are_found(tmp_path, old, new, what):
    src = open(os.path.join(CSRC, "kv_index.hpp")).read()
    assert src.count(old) == 1
    (tmp_path / "kv_index.hpp").write_text(src.replace(old, new))
    r = _run(tmp_path, str(tmp_path))
    assert r.returncode != 0 and what in r.stdout, r.stdout
