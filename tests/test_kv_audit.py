"""CPU audit of the paged cache's index arithmetic (no GPU): tests/kv_audit.hip enumerates the functions of
csrc/kv_index.hpp that the append and attention kernels use; planted mistakes (in a copy) make it fail."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_precision_row_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


def _run(tmp_path, include):
    exe = str(tmp_path / "kv_audit")
    b = subprocess.run([HIPCC, "-std=c++17", "-O1", "-x", "hip", "--cuda-host-only", "-I" + include, "-I" + CSRC,
                        os.path.join(ROOT, "tests", "kv_audit.hip"), "-o", exe], capture_output=True, text=True)
    assert b.returncode == 0, b.stdout + b.stderr
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


def test_every_page_and_piece_is_in_bounds(tmp_path):
    r = _run(tmp_path, CSRC)
    assert r.returncode == 0 and r.stdout.startswith("ok:"), r.stdout[-1000:]


@pytest.mark.parametrize("old,new", [
    ("return id < 0 || id >= c.num_pages ? -1 : id;", "return id;"),                          # a table entry trusted
    ("+ 2 * (int64_t)b;", "+ (int64_t)b;"),                                                   # too few slots
    ("hi = hi < lo ? lo : (hi > t ? t : hi);", "hi = hi < lo ? lo : hi;"),                    # rows past T
    ("if (r.n == 0 || past < 0) return none;", "if (r.n == 0) return none;"),                 # a negative position
    ("(unsigned)total + (unsigned)target - 1) / (unsigned)target", "(unsigned)total) / (unsigned)target"),
    ("2 * (int64_t)r + (at_begin ? 0 : 1)", "(int64_t)r"),
    ("lo = lo / kTile * kTile;", ""),
    ("if (hi > room) hi = room;", ""),
    ("if (D == 64) return gran;", "if (D == 64) return token & 3;"),                          # a bank conflict
    ("return token * D + 16 * (piece ^ k_flip<D, kind>(token));", "return token * D + 16 * piece;"),
    ("(c << run) + ((g & in) ^ (c << run >> 4))", "(c << run) + (g & in)"),
])
def test_planted_mistakes_are_found(tmp_path, old, new):
    src = open(os.path.join(CSRC, "kv_index.hpp")).read()
    assert src.count(old) >= 1
    (tmp_path / "kv_index.hpp").write_text(src.replace(old, new))
    r = _run(tmp_path, str(tmp_path))
    assert r.returncode != 0, r.stdout
