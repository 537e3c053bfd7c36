"""Which device the library's calls are made on, without a GPU: a child process
loads tests/fake_hip.c in the HIP runtime's place (it only writes down each
call and the device current at it). A handle made on one device is used and
freed while another one is current: with a NULL stream, everything that reaches
a device must be done on the handle's own, and the caller's device be current
again afterwards."""
import os
import subprocess
import sys

import pytest

import sparse_moe_gemm_amd as cm

HERE = os.path.dirname(os.path.abspath(__file__))

CHILD = """
import ctypes, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
fake.fake_log.restype = ctypes.c_char_p
sys.path.insert(0, sys.argv[2])
import sparse_moe_gemm_amd as cm
flags, timing = int(sys.argv[3]), cm.FLAG_STAGE_TIMING
P = 0x100000

def device():
    d = ctypes.c_int(-1)
    fake.hipGetDevice(ctypes.byref(d))
    return d.value

def step(name, fn):
    fake.fake_clear()
    st = fn()
    assert st == cm.OK, (name, st)
    for line in fake.fake_log().decode().splitlines():
        print(name, line)
    print(name, "current", device(), 0)

fake.hipSetDevice(1)
st, h = cm.colibri_moe_init(cm.Config(256, 256, 8, 2, 64, cm.BF16, flags | timing), cm.Weights(P, P, P, P, P))
assert st == cm.OK, st
fake.hipSetDevice(0)
step("forward", lambda: cm.colibri_moe_forward(h, P, 64, P))
step("static", lambda: cm.colibri_moe_forward_static(h, P, 64, P))
step("few", lambda: cm.colibri_moe_forward_few(h, P, 4, P))
step("free", lambda: cm.colibri_moe_free(h))
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("fake") / "libfakehip.so")
    subprocess.run(["gcc", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", os.path.join(HERE, "fake_hip.c"), "-o", so],
                   check=True)
    return so


@pytest.mark.parametrize("flags", [0, cm.FLAG_FP8_WEIGHTS, cm.FLAG_MXFP4_WEIGHTS | cm.FLAG_MXFP4_ACTIVATIONS])
def test_calls_are_made_on_the_handles_device(fake, flags):
    r = subprocess.run([sys.executable, "-c", CHILD, fake, os.path.dirname(HERE), str(flags)], capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    lines = [line.split() for line in r.stdout.splitlines()]
    wrong = [v for v in lines if v[2] != ("0" if v[1] == "current" else "1")]
    assert not wrong, wrong
    seen = {(v[0], v[1]) for v in lines}
    for call in ("forward", "static", "few"):
        assert {(call, w) for w in ("launch", "record", "synchronize", "current")} <= seen
    assert {("free", w) for w in ("synchronize", "free", "destroy", "current")} <= seen
