"""Buffers of one call that overlap, without a GPU (tests/fake_hip.c stands in for the
runtime and runs nothing): rms_norm takes outputs in an input's place and refuses
every other overlap, against the sets of bytes themselves; int4_linear takes no y that
overlaps what it reads."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

SETUP = """
import ctypes, random, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
import sparse_moe_gemm_amd as cm
P = 0x100000
"""

NORM = SETUP + """
NAMES = ("x", "residual", "y", "residual_out", "codes", "scales")

def call(rows, cols, dtype, place, weight=P + (1 << 20), wdtype=None):
    fake.fake_clear()
    at = {n: place.get(n, (None, cols)) for n in NAMES}
    return cm.colibri_moe_rms_norm(cm.Norm(
        at["x"][0], at["x"][1], at["residual"][0], at["residual"][1], weight, dtype, dtype if wdtype is None else wdtype,
        rows, cols, 1e-6, at["y"][0], at["residual_out"][0], at["residual_out"][1], at["codes"][0], at["scales"][0]))

def held(name, rows, cols, es, place):
    if name not in place:
        return set()
    p, stride = place[name]
    if name == "scales":
        return set(range(p, p + 4 * rows))
    size = 1 if name == "codes" else es
    if name in ("y", "codes"):
        stride = cols
    return {p + r * stride * size + b for r in range(rows) for b in range(cols * size)}

rng = random.Random(1)
seen = {cm.OK: 0, cm.ERR_INVALID_ARG: 0}
for turn in range(60000):
    es = rng.choice((2, 4))
    rows, cols = rng.randint(1, 7), rng.randint(1, 9)
    wide = rng.choice((0, 0, 4, 20, 90))
    def spot():
        return P + es * rng.randint(0, rng.choice((4, 40, 400)))
    strides = [cols, cols + rng.randint(0, wide), cols + rng.randint(0, wide)]
    place = {"x": (spot(), rng.choice(strides)), "y": (spot(), cols)}
    if rng.random() < 0.5:
        place["residual"] = (spot(), rng.choice(strides))
    if rng.random() < 0.5:
        place["residual_out"] = (spot(), rng.choice(strides))
    if rng.random() < 0.3:
        place["codes"], place["scales"] = (P + rng.randint(0, 2000), cols), (P + 4 * rng.randint(0, 500), 1)
    for out in ("y", "residual_out"):  # in an input's place, now and then
        if out in place and rng.random() < 0.4:
            src = rng.choice([n for n in ("x", "residual") if n in place])
            place[out] = place[src] if out == "residual_out" else (place[src][0], cols)
    weight = spot() if rng.random() < 0.2 else P + (1 << 20)
    bytes_ = {n: held(n, rows, cols, es, place) for n in place}
    bytes_["weight"] = set(range(weight, weight + cols * es))
    bad = False
    outs = [n for n in ("y", "residual_out", "codes", "scales") if n in place]
    for o in outs:
        for n in bytes_:
            if n == o or not bytes_[o] & bytes_[n]:
                continue
            alike = (o in ("y", "residual_out") and n in ("x", "residual") and place[o][0] == place[n][0]
                     and (rows == 1 or place[o][1] == place[n][1]))
            bad = bad or not alike
    st = call(rows, cols, cm.BF16 if es == 2 else cm.F32, place, weight)
    want = cm.ERR_INVALID_ARG if bad else cm.OK
    assert st == want, (turn, st, want, rows, cols, es, place, weight)
    seen[st] += 1
print("seen", seen[cm.OK], seen[cm.ERR_INVALID_ARG])

# long calls: column slices of one buffer, side by side and one value too near
n, d = 1 << 20, 512
row = (P, 2 * d)
assert call(n, d, cm.BF16, {"x": row, "residual_out": (P + 2 * d, 2 * d)}, weight=1 << 44) == cm.OK
assert call(n, d, cm.BF16, {"x": row, "residual_out": (P + 2 * d - 2, 2 * d)}, weight=1 << 44) == cm.ERR_INVALID_ARG
assert call(n, d, cm.BF16, {"x": row, "residual_out": (P - 2 * d + 2, 2 * d)}, weight=1 << 44) == cm.ERR_INVALID_ARG
assert call(n, d, cm.BF16, {"x": row, "y": (P + n * 4 * d - 2 * d, d)}, weight=1 << 44) == cm.OK
assert call(n, d, cm.BF16, {"x": row, "y": (P + n * 4 * d - 2 * d - 2, d)}, weight=1 << 44) == cm.ERR_INVALID_ARG
"""


LINEAR = SETUP + """
m = cm.Int4(4, 64, 256, 128, cm.BF16, 0)  # y [4][2][64] bf16: 1024 bytes
SIZES = dict(packed=cm.colibri_moe_int4_bytes(m), x=2048, ids=32, weights=32)

def call(y, summed=False, **at):
    fake.fake_clear()
    p = {n: 0x1000000 * (i + 2) for i, n in enumerate(SIZES)}
    p.update(at)
    return cm.colibri_moe_int4_linear(m, p["packed"], p["x"], 4, 2, 0, p["ids"], p["weights"] if summed else None, y,
                                      cm.BF16)

for name, size in SIZES.items():
    for summed in (False, True):
        if name == "weights" and not summed:
            continue
        wide = 512 if summed else 1024
        for at, want in ((P, cm.ERR_INVALID_ARG), (P + wide - 16, cm.ERR_INVALID_ARG), (P + wide, cm.OK),
                         (P - size + 16, cm.ERR_INVALID_ARG), (P - size, cm.OK)):
            assert call(P, summed, **{name: at}) == want, (name, summed, at - P)
print("done")
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("fake") / "libfakehip.so")
    subprocess.run(["gcc", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", os.path.join(HERE, "fake_hip.c"), "-o", so],
                   check=True)
    return so


def child(fake, program):
    r = subprocess.run([sys.executable, "-c", program, fake, os.path.dirname(HERE)], capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_rms_norm(fake):
    _, taken, refused = child(fake, NORM).split()
    assert int(taken) > 5000 and int(refused) > 5000


def test_int4_linear(fake):
    assert child(fake, LINEAR).split() == ["done"]
