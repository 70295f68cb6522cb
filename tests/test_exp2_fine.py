"""The degree-5 exp2 of the FMA pipe (exp2_fine2 in csrc/sm100.cuh), which serves fp32 outputs.

CPU: the constants compiled into the kernels are the fp32 roundings of the fit that
token_skipping_sparse_b200/exp2_poly_fit.py derives, and its error is that of fp32 rounding."""

import importlib.util
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_fine_constants_are_the_fit():
    spec = importlib.util.spec_from_file_location(
        "exp2_poly_fit", os.path.join(ROOT, "token_skipping_sparse_b200", "exp2_poly_fit.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    want = m.fit_fine().astype(np.float32)[::-1]
    src = open(os.path.join(ROOT, "token_skipping_sparse_b200", "csrc", "sm100.cuh")).read()
    body = src[src.index("void exp2_fine2("):]
    body = body[:body.index("\n}\n")]
    consts = [float(v) for v in re.findall(r"f2pack\(([0-9.e+-]+)f, \1f\)", body)]
    # the shifter 1.5 * 2^23 and its negative, the -1, then c5 .. c0 in Horner order
    poly = [v for v in consts if abs(v) < 2.0 and v != -1.0]
    assert np.array_equal(np.asarray(poly, dtype=np.float32), want), (poly, want)
    f = np.linspace(-0.5, 0.5, 100001, dtype=np.float32)
    err = np.abs(m.horner_fp32(want[::-1], f).astype(np.float64) / 2.0 ** f.astype(np.float64) - 1.0).max()
    # half a step of the sum (2^-24), the products' roundings and the fit: within 2^-21.8
    assert err < 2.7e-7
