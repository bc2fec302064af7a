"""Kernel selection and launch geometry of the dropout calls, checked on the
host (no GPU), and that the library holds no dropout kernel that no call
reaches.

``tests/dropout_geometry.cu`` is compiled with nvcc against the library's own
selection headers and visits every row length of every type and variant."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "dropout_geometry.cu")
TYPES = {"f": "f32", "13__nv_bfloat16": "bf16", "6__half": "f16"}


@pytest.fixture(scope="module")
def run():
    from layernorm_fwd_bwd_b200 import build
    exe = os.path.join(build.BUILD_DIR, "dropout_geometry")
    deps = [SRC, *build.DEPENDS]
    if not os.path.exists(exe) or any(os.path.getmtime(d) > os.path.getmtime(exe)
                                      for d in deps):
        os.makedirs(build.BUILD_DIR, exist_ok=True)
        subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-o", exe, SRC], check=True,
                       capture_output=True, text=True)
    return subprocess.run([exe], capture_output=True, text=True)


def test_no_check_fails(run):
    fails = [l for l in run.stdout.splitlines() if l.startswith("FAIL")]
    assert run.returncode == 0 and not fails, "\n".join(fails[:20]) + run.stderr
    last = run.stdout.splitlines()[-1].split()
    assert last[0] == "checks" and int(last[1]) > 1000000 and last[3] == "0"


def built():
    """The ring, split and ragged kernels with dropout that the objects hold, as
    the geometry check names them."""
    from layernorm_fwd_bwd_b200 import build
    build.build()
    if not all(os.path.exists(build.ptxas_report(o)) for o in build.objects()):
        build.build(force=True)      # a library built before reports were kept
    out = set()
    name = re.compile(r"Compiling entry function '_ZN3lnk\d+ln_(fwd_ragged|bwd_ragged|bwd_tma|"
                      r"bwd_split)_kernelI(f|13__nv_bfloat16|6__half)((?:L[ib]\d+E)+)E")
    for obj in build.objects():
        for kernel, t, args in name.findall(open(build.ptxas_report(obj)).read()):
            a = [int(v) for v in re.findall(r"L[ib](\d+)E", args)]
            head = f"{kernel} {TYPES[t]}"
            if kernel == "fwd_ragged":                       # V, L, GROUPS
                out.add(f"{head} {a[0]} {a[1]} {a[2]}")
            elif a[-1] < 4:                                  # MODE without dropout
                continue
            elif kernel == "bwd_ragged":                     # V, L, GROUPS, MODE
                out.add(f"{head} {a[3]} {a[0]} {a[1]} {a[2]}")
            elif kernel == "bwd_tma":                        # V, NC, S, RR, W, MODE
                out.add(f"{head} {a[5]} {a[0]} {a[4]}")
            else:                                            # VR, VC, NR, NCOL, MODE
                out.add(f"{head} {a[4]} {a[0]} {a[1]}")
    return out


def test_every_dropout_kernel_is_reached(run):
    """The kernels in the library are exactly those that the selection
    reaches."""
    used = {l[4:] for l in run.stdout.splitlines() if l.startswith("use ")}
    have = built()
    assert len(used) > 200
    assert have - used == set(), sorted(have - used)
    assert used - have == set(), sorted(used - have)
