"""A launch that fails ends its call: nothing is queued behind it that would read what it has not written.  In a process of
its own, with a launch call of the test's in front of the runtime's, so that no device is needed."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import ctypes as C, sys
stub, lib, good = C.CDLL(sys.argv[1], C.RTLD_GLOBAL), C.CDLL(sys.argv[2]), int(sys.argv[3])
count, passes = (C.c_int.in_dll(stub, "bllm_test_" + x) for x in ("launches", "good"))
P, i64, f64, size = C.c_void_p(4096), C.c_int64, C.c_double, C.c_size_t(1 << 40)
def calls():
    pages = (1, i64(9), i64(64))  # bf16 pages
    heads = (i64(4), i64(2), i64(64))
    yield "attention", 2, lib.bllm_attention(P, P, P, 1, P, P, i64(1), i64(8), i64(8192), *heads, i64(256), i64(128), i64(128),
                                             f64(1.0), 1, i64(0), f64(0.0), None, None, P, P, size, None)
    yield "step", 2, lib.bllm_attention_step(P, 1, i64(1), *heads, i64(256), P, P, None, None, *pages, P, i64(128), P,
                                             f64(1.0), i64(0), f64(0.0), None, None, P, P, size, None)
    yield "write", 1, lib.bllm_kv_write(P, P, 1, P, i64(1), i64(8), i64(2), i64(64), i64(128), i64(128), None, P, i64(4),
                                        *pages, P, P, None, None, None)
    # more workgroups than one launch has threads for
    yield "many", 2, lib.bllm_attention(P, P, P, 1, P, P, i64(65535), i64(1 << 26), i64(1 << 26), i64(1024), i64(1024), i64(8), i64(8192),
                                        i64(8192), i64(8192), f64(1.0), 1, i64(0), f64(0.0), None, None, P, P, size, None)
it = calls()
while True:
    count.value, passes.value = 0, good
    try:
        name, most, rc = next(it)
    except StopIteration:
        break
    print(name, most, count.value, rc)
"""


@pytest.mark.parametrize("good", [0, 1, 1000000])
def test_a_failed_launch_ends_its_call(tmp_path, good):
    import byte_level_lm_amd as B
    from byte_level_lm_amd import _lib
    B.lib()
    stub = str(tmp_path / "launches.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-o", stub, os.path.join(ROOT, "tests", "c_abi", "launches.cpp")], check=True)
    out = subprocess.run([sys.executable, "-c", PROGRAM, stub, _lib.LIB_PATH, str(good)], capture_output=True, text=True,
                         timeout=120, check=True).stdout
    rows = [line.split() for line in out.splitlines()]
    assert [r[0] for r in rows] == ["attention", "step", "write", "many"]
    for name, most, count, rc in ((r[0], *map(int, r[1:])) for r in rows):
        if good < most:
            assert (count, rc) == (good + 1, -4), name
        else:
            assert rc == 0 and (count == most or name == "many" and count > most), name
