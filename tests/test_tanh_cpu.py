"""The packed kernels' FMA-pipe tanh on the CPU: the constants in csrc/tanh_poly.cuh are the ones the
committed Remez generator produces, and an f32 emulation of the device function stays within 2e-7 of
tanh, relative, up to the limit beyond which the kernels do not take it."""
import importlib.util
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "causal_flash_attention_attn_b200", "csrc")


def generator():
    spec = importlib.util.spec_from_file_location("gen_tanh_poly", os.path.join(CSRC, "gen_tanh_poly.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def device_coefficients():
    text = open(os.path.join(CSRC, "tanh_poly.cuh")).read()
    body = text[text.index("uint64_t tanh_poly2"):]
    body = body[:body.index("\n}\n")]
    pairs = re.findall(r"f2_make\((-?[0-9.e+-]+)f, (-?[0-9.e+-]+)f\)", body)
    assert len(pairs) == 6 and all(a == b for a, b in pairs)
    return np.array([float(a) for a, _ in reversed(pairs)], dtype=np.float32)  # c0 .. c5


def test_constants_are_the_generators():
    gen = generator()
    err, c32 = gen.f32_error(gen.remez_rel(5))
    assert err < 2e-7
    np.testing.assert_array_equal(c32, device_coefficients())
    text = open(os.path.join(CSRC, "tanh_poly.cuh")).read()
    assert float(re.search(r"kTanhPolyLimit = ([0-9.]+)f", text).group(1)) == gen.LIMIT


def test_emulated_device_tanh_within_the_bound():
    c = device_coefficients()
    y = np.concatenate([np.linspace(-0.75, 0.75, 1000001), [1e-30, -1e-30, 1e-6]]).astype(np.float32)
    u = (y * y).astype(np.float32)
    p = np.full_like(y, c[5])
    for k in range(4, -1, -1):  # fused multiply-adds: one rounding
        p = (p.astype(np.float64) * u + c[k]).astype(np.float32)
    got, ref = (p * y).astype(np.float64), np.tanh(y.astype(np.float64))
    live = ref != 0
    assert np.max(np.abs(got[live] / ref[live] - 1)) < 2e-7 and np.all(got[~live] == 0)
