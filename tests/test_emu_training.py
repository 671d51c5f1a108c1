"""The unchanged kernels of the balance losses and the update of the parameters
on the CPU (see test_cpu_emu), under AddressSanitizer: every global-memory access
is bounds-checked against arrays of exactly the promised extents, and the
outputs pass the fp64 oracle's checks.  LRM_EMU_FULL=1 runs every case."""

from __future__ import annotations

import concurrent.futures as cf
import os
import struct
import subprocess

import numpy as np
import pytest
import torch

import training_cases as TC
from test_cpu_emu import CLANG, CSRC, EMU, FLAGS, ROOT
from test_emu_forward import _raw, call, stored

FULL = bool(os.environ.get("LRM_EMU_FULL"))


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("clang++ of the ROCm toolchain not found")
    out = tmp_path_factory.mktemp("emu_training")

    def compile_one(src):
        obj = os.path.join(out, os.path.basename(src) + ".o")
        r = subprocess.run([CLANG, *FLAGS, "-DLRM_CPU_EMU", "-x", "c++", "-I", EMU, "-I",
                            os.path.join(ROOT, "include"), "-I", CSRC, "-c", src, "-o", obj],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{src}:\n{r.stderr[-4000:]}")
        return obj

    srcs = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        objs = list(ex.map(compile_one, srcs + [os.path.join(EMU, "emu_training.cpp")]))
    exe = os.path.join(out, "emu_training")
    r = subprocess.run([CLANG, "-fsanitize=address", "-o", exe, *objs, "-lpthread"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    return exe


def bits(x):
    """A float64 as the int64 that holds it."""
    return struct.unpack("<q", struct.pack("<d", float(x)))[0]


class Number(np.ndarray):
    """Numbers between the arrays: no byte count before them."""


def numbers(*v):
    return np.array(v, np.int64).view(Number)


@pytest.fixture
def run(driver, tmp_path, monkeypatch):
    import test_emu_forward as EF
    monkeypatch.setattr(EF, "_raw", lambda v: v.tobytes() if isinstance(v, Number) else _raw(v))
    return lambda nums, arrays, outs: call(driver, tmp_path, nums, arrays, outs)


def balance_nums(op, c, *more):
    S = 1 if c["seq"] is None else len(c["seq"]) - 1
    return [op, c["T"], c["E"], c["k"], int(c["score"] == "sigmoid"), int(c["renorm"]),
            int(c["dtype"] == "bf16"), c["ld"] or c["E"], S, *more]


def balance_arrays(c):
    seq = None if c["seq"] is None else torch.tensor(c["seq"], dtype=torch.int32)
    return [numbers(bits(c["coef"]), bits(c["z_coef"])), stored(dict(c, ld=c["ld"] or c["E"])),
            c["expert_mask"], c["token_mask"], c["expert"], c["counts_in"], seq]


BAL = sorted(TC.BALANCE) if FULL else ["seqs", "one_seq", "sigmoid_low", "twice", "strided"]


@pytest.mark.parametrize("name", BAL)
def test_balance(run, name):
    c = TC.balance_case(name)
    S, E, T = 1 if c["seq"] is None else len(c["seq"]) - 1, c["E"], c["T"]
    outs = [((2,), torch.float32), ((S * E + 2,), torch.float32)]
    if c["counts_in"] is None:
        outs.append(((S, E), torch.int32))
    got = run(balance_nums(0, c), balance_arrays(c), outs)
    TC.check_balance(c, *got)
    # rows two elements further apart than they are long; what lies between stays
    dt, ldd = TC.DT[c["dtype"]], E + 2
    n = (T - 1) * ldd + E
    es = torch.empty(0, dtype=dt).element_size()
    d = run(balance_nums(1, c, n * es, ldd), balance_arrays(c) + [got[1], c["dloss"], c["dweight"]],
            [((n,), dt)])[0]
    pad = torch.cat([d, torch.full(((T * ldd - n) * es,), 0xCD, dtype=torch.uint8).view(dt)]).view(T, ldd)
    TC.check_balance_bwd(c, pad[:, :E])
    assert (pad[:, E:].contiguous().view(torch.uint8) == 0xCD).all()


@pytest.mark.parametrize("S,counts", [(1, False), (1, True), (3, False)])
def test_balance_without_tokens(run, S, counts):
    """No tokens, and no logits: nothing is read."""
    E, k = 8, 2
    c = torch.ones(S, E, dtype=torch.int32) if counts else None
    seq = torch.zeros(S + 1, dtype=torch.int32) if S > 1 else None
    nums = [0, 0, E, k, 0, 1, 0, E, S]
    arrays = [numbers(bits(0.5), bits(0.25)), None, None, None, None if counts else
              torch.empty(0, dtype=torch.int32), c, seq]
    outs = [((2,), torch.float32), ((S * E + 2,), torch.float32)]
    if not counts:
        outs.append(((S, E), torch.int32))
    got = run(nums, arrays, outs)
    assert got[0].tolist() == [0.0, 0.0] and got[1].tolist() == [0.0] * (S * E) + [0.5, 0.5]
    assert counts or not got[2].any()
    nums[0] = 1
    run(nums + [-1, E], arrays + [got[1], None, None], [])


PAR = sorted(TC.PARAMS) if FULL else ["odd_f32", "eight_bf16", "unaligned_eight", "master", "forty"]


@pytest.mark.parametrize("name", PAR)
@pytest.mark.parametrize("on_device", [False, True])
def test_params(run, name, on_device):
    if on_device and not FULL and name != "eight_bf16":
        pytest.skip("extended emulation case (set LRM_EMU_FULL=1)")
    c = TC.param_case(name)
    t = c["t"]
    eight = c["bits"] == 8
    nums = [2, len(t), int(c["p"] == "bf16"), int(c["g"] == "bf16"), int(eight), int(c["master"]),
            c["offset"], int(c["clip"])]
    lr = 7.0 if on_device else c["lr"]
    arrays = [numbers(*(bits(x) for x in (lr, c["beta1"], c["beta2"], c["eps"], c["scale"],
                                          c["max_norm"])), 1 if on_device else c["step"], c["seed"])]
    outs = []
    for i, q in enumerate(t):
        arrays.append(numbers(q["n"], bits(c["lrs"][i]), bits(c["decays"][i])))
        for key in ("g", "p", "master", "m", "v", "m_exp", "v_exp"):
            arrays.append(q[key])
            if key != "g" and q[key] is not None:
                outs.append((tuple(q[key].shape), q[key].dtype))
    if on_device:  # (the rate in fp32)
        c["lr"] = float(np.float32(c["lr"]))
        arrays += [torch.tensor([c["lr"]]), torch.tensor([c["step"] - 1])]
        outs.append(((1,), torch.int64))
    else:
        arrays += [None, None]
    outs.append(((1,), torch.float64))
    got = run(nums, arrays, outs)
    assert abs(float(got[-1][0]) - c["sumsq"]) <= 1e-13 * c["sumsq"]
    if on_device:
        assert int(got[-2][0]) == c["step"]
    it = iter(got)
    TC.check_adamw(c, [{k: next(it) if q[k] is not None else None
                        for k in ("p", "master", "m", "v", "m_exp", "v_exp")} for q in t])


@pytest.mark.parametrize("second", [0, 1])
@pytest.mark.parametrize("dtype,skip", [("bf16", 0), ("f32", 5)])
def test_moment_read(run, second, dtype, skip):
    n = 300
    codes = torch.arange(n).to(torch.uint8)
    exps = torch.tensor([(37 * i) % 200 + 40 for i in range(10)], dtype=torch.uint8)
    dt = TC.DT[dtype]
    got = run([3, n, second, int(dtype == "bf16"), skip, n * (2 if dtype == "bf16" else 4)],
              [codes, exps], [((n,), dt)])[0]
    assert torch.equal(got.double(), torch.as_tensor(TC.values(codes.numpy(), exps.numpy(), second)))
