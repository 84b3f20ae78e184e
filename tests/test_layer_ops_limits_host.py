"""Limits of the operators of a trained layer: where one begins to refuse, and that what a launch cuts into parts has its
place in the workspace (nothing reaches a device)."""

from __future__ import annotations

import ctypes as C
import os
import shutil
import subprocess

import pytest

import muon_newton_schulz_step_amd as M
from test_layer_ops_host import _route_opt
from test_train_ops_host import BASE, BIG, _expect

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "muon_newton_schulz_step_amd", "csrc")


def test_route_refuses_from_its_limit_of_tokens_on():
    far = 1 << 50  # apart from each other at any of these sizes
    for n, e, k in ((1 << 26, 257, 1), (1 << 30, 8, 2), (1 << 31, 1, 1)):
        _expect("muon_route", "MUON_ERR_UNSUPPORTED", BASE, n, e, e, 0, None, None, _route_opt(groups=1), BASE + far, 0, k,
                BASE + 2 * far, None)
        _expect("muon_route_backward", "MUON_ERR_UNSUPPORTED", BASE, n, e, e, 0, None, _route_opt(groups=1), BASE + far, 0, k,
                BASE + 2 * far, BASE + 3 * far, e, 1, None)
    assert BIG < far


def test_parts_fit_the_workspace(tmp_path):
    # tests/host/linear_parts.cpp goes through the launches' rules and the workspace's
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not available")
    exe = str(tmp_path / "linear_parts")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, os.path.join(ROOT, "tests", "host", "linear_parts.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "linear parts ok" in r.stdout, r.stdout[-2000:]
    assert int(r.stdout.split("launches, ")[1].split()[0]) > 1000  # many of them in parts


def test_the_library_asks_for_that_workspace():
    # few rows by long weights: 32 parts of fp32 sums; many rows: none
    assert M.linear_workspace_bytes(4, 16384, 512, 1) >= 256 + 32 * 4 * 512 * 4
    assert M.linear_workspace_bytes(8192, 4096, 11008, 1) == 256


def test_products_refuse_from_their_limit_of_tiles_on():
    # of 128 x 128 elements; a grid of 64 columns a workgroup has 2^32 threads from 2^30 - 63 columns on
    n = C.c_size_t()
    for f in ("muon_linear_workspace_bytes", "muon_linear_weight_grad_workspace_bytes"):
        for rows, a, b, groups in ((1, 1, (1 << 30) - 64, 1), (1, (1 << 30) - 64, 1, 1), (1 << 20, 1 << 17, 8, 1), (1 << 20, 8, 1 << 17, 1),
                                   (8, 1 << 13, 1 << 14, 1024)):
            _expect(f, "MUON_ERR_UNSUPPORTED", rows, a, b, groups, C.byref(n))
    for f in (M.linear_workspace_bytes, M.linear_weight_grad_workspace_bytes):
        assert f(1, 1, (1 << 30) - 129, 1) >= 256 and f((1 << 20) - 256, (1 << 17) - 128, 8, 1) >= 256
