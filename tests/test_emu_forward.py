"""The unchanged kernels of the router, the experts' forward pass and its
epilogue's backward pass on the CPU (see test_cpu_emu), under
AddressSanitizer: every global-memory access is bounds-checked against arrays
of exactly the promised extents, and the outputs pass the fp64 oracle's
checks.  LRM_EMU_FULL=1 runs every case of the GPU tests that fits."""

from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess

import numpy as np
import pytest
import torch

import forward_cases as FC
from test_cpu_emu import CLANG, CSRC, EMU, FLAGS, ROOT, _sources

FULL = bool(os.environ.get("LRM_EMU_FULL"))
# inputs of more bytes than this are packed before the product (2 GiB in the
# product build; lowered here so that some of the small cases pack)
GATHER_MAX = 20000


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("clang++ of the ROCm toolchain not found")
    out = tmp_path_factory.mktemp("emu_forward")

    def compile_one(src):
        obj = os.path.join(out, os.path.basename(src) + ".o")
        r = subprocess.run([CLANG, *FLAGS, "-DLRM_CPU_EMU", f"-DLRM_FWD_GATHER_MAX={GATHER_MAX}", "-x", "c++", "-I", EMU, "-I",
                            os.path.join(ROOT, "include"), "-I", CSRC, "-c", src, "-o", obj],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{src}:\n{r.stderr[-4000:]}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        objs = list(ex.map(compile_one, _sources() + [os.path.join(EMU, "emu_forward.cpp")]))
    exe = os.path.join(out, "emu_forward")
    r = subprocess.run([CLANG, "-fsanitize=address", "-o", exe, *objs, "-lpthread"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    return exe


def _raw(v) -> bytes:
    if v is None:
        return np.int64(-1).tobytes()
    if isinstance(v, torch.Tensor):
        v = v.contiguous()
        v = (v.view(torch.int16) if v.dtype == torch.bfloat16 else v).numpy()
    b = np.ascontiguousarray(v).tobytes()
    return np.int64(len(b)).tobytes() + b


def call(exe, tmp_path, nums, arrays, outs, expect=(0, 0), env_extra=None):
    """outs: [(shape, dtype)] in the driver's order; returns CPU tensors that
    held bytes 0xCD before the call."""
    h = np.zeros(32, np.int64)
    h[:len(nums)] = nums
    fin, fout = tmp_path / "in.bin", tmp_path / "out.bin"
    fin.write_bytes(h.tobytes() + b"".join(_raw(a) for a in arrays))
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1")
    env.pop("LRM_FWD_TILE", None)
    env.update(env_extra or {})
    res = subprocess.run([exe, str(fin), str(fout)], capture_output=True, text=True, timeout=600,
                         env=env)
    assert res.returncode == 0, f"emulated run failed ({res.returncode}):\n{res.stderr[-6000:]}"
    buf = fout.read_bytes()
    status = tuple(int(v) for v in np.frombuffer(buf, np.int32, 2))
    assert status == tuple(expect), status
    got, off = [], 8
    for shape, dt in outs:
        n = int(np.prod(shape)) * torch.empty(0, dtype=dt).element_size()
        raw = torch.from_numpy(np.frombuffer(buf, np.uint8, n, off).copy())
        got.append(raw.view(dt).reshape(shape) if n else torch.empty(shape, dtype=dt))
        off += n
    assert off == len(buf)
    return got


def nbytes(shape, dt):
    return int(np.prod(shape)) * torch.empty(0, dtype=dt).element_size()


def held(shape, dt):
    n = nbytes(shape, dt)
    raw = torch.full((n,), 0xCD, dtype=torch.uint8)
    return raw.view(dt).reshape(shape) if n else torch.empty(shape, dtype=dt)


def router_nums(op, c):
    return [op, c["T"], c["E"], c["k"], int(c["score"] == "sigmoid"), int(c["renorm"]), c["n_group"],
            c["topk_group"], int(c["group_rule"] == "top2"), int(c["scale"] * 1024),
            int(c["dtype"] == "bf16"), c["ld"]]


def stored(c):
    """The logits with the rows c['ld'] apart, ending with the last row's last element."""
    T, E, ld = c["T"], c["E"], c["ld"]
    flat = torch.zeros((T - 1) * ld + E, dtype=c["logits"].dtype)
    for t in range(T):
        flat[t * ld:t * ld + E] = c["logits"][t]
    return flat


SMALL_ROUTE = ["t1", "odd", "ties_bias", "equal_bias", "groups_top2", "groups_softmax",
               "masks_groups", "lowest_sigmoid", "widest_groups", "strided"]


@pytest.mark.parametrize("name", list(FC.ROUTE_CASES) if FULL else SMALL_ROUTE)
def test_emu_route(driver, tmp_path, name):
    c = FC.route_case(name)
    n = c["T"] * c["k"]
    i32 = torch.int32
    e, w, t, cnt = call(driver, tmp_path, router_nums(0, c) + [4 * n, 4 * n, 4 * c["E"]],
                        [stored(c), c["bias_t"], c["emask"], c["tmask"]],
                        [((n,), i32), ((n,), torch.float32), ((n,), i32), ((c["E"],), i32)])
    FC.judge_route(c, e, w, t, cnt)


@pytest.mark.parametrize("name", list(FC.ROUTE_CASES) if FULL else
                         ["odd", "odd_bf16", "masks_softmax", "wide", "strided"])
def test_emu_route_bwd(driver, tmp_path, name):
    c = FC.route_case(name)
    e, dw = FC.route_grad_inputs(c, name)
    T, E = c["T"], c["E"]
    ldd = E + (3 if name in ("odd", "strided") else 0)
    dt = c["logits"].dtype
    n = (T - 1) * ldd + E
    got, = call(driver, tmp_path, router_nums(1, c) + [nbytes((n,), dt), ldd],
                [stored(c), c["bias_t"], c["emask"], c["tmask"], e, dw], [((n,), dt)])
    rows = torch.stack([got[t * ldd:t * ldd + E] for t in range(T)])
    FC.judge_route_bwd(c, e, dw, rows)
    gap = torch.cat([got[t * ldd + E:(t + 1) * ldd] for t in range(T - 1)] or [got[:0]])
    assert (gap.view(torch.uint8) == 0xCD).all()


@pytest.mark.parametrize("T,k,e0,E", [(1, 1, 0, 1), (300, 3, 4, 5), (3001, 2, 2, 3), (50, 4, 90, 8)])
def test_emu_share(driver, tmp_path, T, k, e0, E):
    from oracle import forward as OF
    rng = np.random.default_rng(T)
    n = T * k
    ex = rng.integers(-1, 12, n).astype(np.int32)
    w = rng.random(n).astype(np.float32)
    i32, f32 = torch.int32, torch.float32
    ot, oe, ow, os_, on = call(driver, tmp_path, [2, T, k, e0, E, 4 * n], [ex, w],
                               [((n,), i32), ((n,), i32), ((n,), f32), ((n,), i32), ((1,), i32)])
    t, e, wr, s = OF.route_share(k, ex, w, e0, E)
    m = int(on[0])
    assert m == s.size
    for got, ref in ((ot, t), (oe, e), (ow, wr), (os_, s)):
        assert np.array_equal(got[:m].numpy(), ref)
        assert (got[m:].view(torch.uint8) == 0xCD).all()


def emu_forward(driver, tmp_path, c, env_extra=None):
    shapes = FC.forward_shapes(c)
    order = ("Y", "Yp", "Z", "A", "B", "h_sumsq")
    pr = c["pairs"]
    nums = [3, c["T"], c["N"], c["E"], int(c["kind"] != "linear"), int(c["dtype"] == "bf16"),
            ("none", "relu", "gelu", "silu").index(c["act"]), c["d_in"], c["d"],
            int(c["x_rows"] == "pair"), c["ldx"], c["d_out"], c["d_in"] * c["d"]]
    nums += [nbytes(*shapes[k]) if k in shapes else -1 for k in order]
    x = c["X_store"].reshape(-1)
    x = x[:x.numel() - (c["ldx"] - c["d_in"])]
    w = [c["W"], c["bias_t"]] if c["kind"] == "linear" else [c["W_gate"], c["W_up"], c["W_down"]]
    got = call(driver, tmp_path, nums, [pr["token"], pr["expert"], pr["weight"], x, c["R"], *w],
               [shapes[k] for k in order if k in shapes], expect=(0, 8 if c["bad"] else 0), env_extra=env_extra)
    got = dict(zip([k for k in order if k in shapes], got))
    FC.judge_forward(c, got, {k: held(*shapes[k]) for k in got})


SMALL_FORWARD = ["lin_one", "lin_one_f32", "lin_odd", "lin_none", "lin_bad", "glu_t1", "glu_t3",
                 "glu_small", "glu_small_f32", "glu_pairs_only", "glu_bad_t1", "lin_no_tokens", "glu_no_tokens", "glu_twice"]


@pytest.mark.parametrize("name", list(FC.FORWARD_CASES) if FULL else SMALL_FORWARD)
def test_emu_forward(driver, tmp_path, name):
    emu_forward(driver, tmp_path, FC.forward_case(name))


@pytest.mark.parametrize("name", ["lin_skew", "lin_odd_f32", "glu_small", "glu_small_f32"])
@pytest.mark.parametrize("tile", ["128", "256"])
def test_emu_forward_tiles(driver, tmp_path, name, tile):
    """The larger tiles on cases small enough to emulate (one that packs its
    input first among them)."""
    emu_forward(driver, tmp_path, FC.forward_case(name), {"LRM_FWD_TILE": tile})


@pytest.mark.parametrize("name", ["lin_none", "lin_no_tokens", "glu_no_tokens", "glu_twice"])
def test_emu_forward_tiles_of_little(driver, tmp_path, name):
    emu_forward(driver, tmp_path, FC.forward_case(name), {"LRM_FWD_TILE": "64"})


@pytest.mark.parametrize("name", list(FC.PAIR_GRAD_CASES) if FULL else
                         ["one", "weights_f32", "no_bias", "gelu", "none_wide", "none_left"])
def test_emu_pair_grad(driver, tmp_path, name):
    c = FC.pair_grad_case(name)
    shapes = FC.pair_grad_shapes(c)
    order = ("dweight", "G", "dbias")
    pr = c["pairs"]
    nums = [4, c["T"], c["N"], c["E"], 0, int(c["dtype"] == "bf16"),
            ("none", "relu", "gelu", "silu").index(c["act"]), 0, c["d"],
            int(c["dy_rows"] == "pair"), c["d"], c["d"], 0]
    nums += [nbytes(*shapes[k]) if k in shapes else -1 for k in order]
    bad = c["bad"] and "dbias" in shapes
    got = call(driver, tmp_path, nums, [pr["token"], pr["expert"], pr["weight"], c["dY"], c["Z"]],
               [shapes[k] for k in order if k in shapes], expect=(0, 8 if bad else 0))
    FC.judge_pair_grad(c, dict(zip([k for k in order if k in shapes], got)))
