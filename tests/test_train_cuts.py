"""Every way in which the training calls cut their products is run by a GPU test (no
GPU needed: the plan's own code is compiled and asked).  A constant of the plan that
changes, or a new shape of tile, shows here as a way that no test takes."""
import math
import os
import random
import shutil
import subprocess

import pytest
import torch

import tests.test_gpu_train as G
from tests.test_gpu_train_cuts import MORE

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = "/opt/rocm"
ACT = {"f32": 0, "bf16": 1}

pytestmark = pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(f"{ROCM}/include/hip"),
                                reason="needs g++ and HIP's headers")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """[(T, H, E, I, k, act, tiles of 256 rows)] -> the ways of each, by call."""
    exe = str(tmp_path_factory.mktemp("plans") / "plans")
    cmd = ["g++", "-std=c++17", "-O2", "-D__HIP_PLATFORM_AMD__", "-I", f"{ROCM}/include", "-I", f"{ROOT}/include",
           f"{ROOT}/tests/train_plans.cpp", f"{ROOT}/sparse_moe_routed_amd/csrc/train_plan.cpp", "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]

    def ask(shapes):
        r = subprocess.run([exe], input="\n".join(" ".join(map(str, s)) for s in shapes), capture_output=True, text=True)
        assert r.returncode == 0
        return [ways(s, *map(int, line.split())) for s, line in zip(shapes, r.stdout.splitlines(), strict=True)]
    return ask


def ways(shape, fits, gs, gp, go, gt, hs, hp, ho, xs, xp, xo, xt, wp, wt, joint):
    """Type, tile shape, split sum, listed tiles, weights read once, cut last tiles: what
    chooses a kernel or how it finds its work."""
    if not fits:
        return {}
    act, listed = shape[5], shape[2] > 64
    dw = "parts" if wp > 1 else "strips" if wp else "wide"
    return dict(save={(act, gs, gp > 1, listed, go if gs < 2 else 0, gt > 1)},
                backward={("dh", act, hs, hp > 1, listed, ho),
                          ("dx", act, xs, xp > 1, listed, xo if xs < 2 and not joint else 0, xt > 1, joint),
                          ("dw", act, dw, wt > 1, joint)})


def named(w, kept):
    """With the form of g and u, which chooses a kernel of the save and of dh."""
    return {("save", *v, kept) for v in w.get("save", ())} | \
           {(*v, kept) if v[0] == "dh" else v for v in w.get("backward", ())}


def drawn(n):
    rng = random.Random(3)
    size = lambda lo, hi: round(math.exp(rng.uniform(math.log(lo), math.log(hi))))
    while n:
        E = rng.choice([1, 1, 1, 2, 3, 5, 8, 9, 16, 33, 64, 65, 70, 100, 128, 256, 512, 1024])
        k = min(E, rng.choice([1, 1, 2, 3, 4, 8, 10]))
        T, H, I = size(1, 20000), 128 * size(1, 40), 32 * size(1, 160)
        if T * max(E, H) < 2 ** 31:
            n -= 1
            per = max(1, T * k // E)
            yield T, H, E, I, k, rng.randint(0, 1), min(E, T * k) * ((per + 255) // 256)


def taken_by_tests(monkeypatch, plans):
    monkeypatch.setattr(G, "DEV", torch.device("cpu"))

    def shape(T, H, E, I, k, act, seed, drop):
        rows = G.Routes(T, E, k, seed, drop).offsets.diff().long()
        return T, H, E, I, k, ACT[act], int(((rows + 255) // 256).sum())

    cases = []                                                  # shape, kept, calls
    for size in G.SIZES:
        for act, kept, _ in G.FORMS:
            cases.append((shape(*size, act, 0, 0.0), kept, ("save", "backward")))
    for act, kept, *size in G.CUTS:
        for seed, call in ((17, "save"), (18, "backward")):
            cases.append((shape(*size, act, seed, 0.1), kept, (call,)))
    for act, *size in MORE:
        for kept in ("act", "8bit"):
            cases.append((shape(*size, act, 19, 0.1), kept, ("save", "backward")))
    taken = set()
    for (_, kept, calls), w in zip(cases, plans([c[0] for c in cases]), strict=True):
        taken |= named({c: w[c] for c in calls}, kept)
    return taken


def test_every_way_is_tested(monkeypatch, plans):
    taken = taken_by_tests(monkeypatch, plans)
    reached = {}
    shapes = list(drawn(120000))
    for s, w in zip(shapes, plans(shapes), strict=True):
        for kept in ("act", "8bit"):
            for v in named(w, kept):
                reached.setdefault(v, s)
    missing = {v: s for v, s in reached.items() if v not in taken}
    assert not missing, missing
    # the draws are dense enough to see nearly all that the tests take
    assert len(taken - set(reached)) <= len(taken) // 20, taken - set(reached)
