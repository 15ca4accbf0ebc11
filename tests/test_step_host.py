"""The host side of E4M3 products, rotations and verification, without a GPU:
bad arguments come back as status codes, and the structures have the header's layout."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import step_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HOST = (ctypes.c_int32 * 4096)()
P = (ctypes.addressof(HOST) + 255) & ~255


def test_fp8_arguments(afx):
    lib, E = afx._lib, afx.AFX_E_ARG
    quantize = lambda x=P, kind=0, xs=128, n=2, cols=128, q=P, qs=128, s=P, ss=2: lib.afx_fp8_quantize(x, kind, xs, n, cols, q, qs, s, ss, None)  # noqa: E731
    assert quantize(n=0) == quantize(cols=0) == afx.AFX_OK
    for bad in ({"kind": 3}, {"n": 1 << 24}, {"cols": 1 << 24}, {"xs": 127}, {"qs": 127}, {"cols": 129, "xs": 200, "qs": 200, "ss": 1}, {"x": None}, {}):
        assert quantize(**bad) == E  # the last: host memory
    product = lambda w=P, ws=128, rows=2, cols=128, x=P, xs=128, xss=2, n=2, kind=2, ys=2: lib.afx_fp8_product(  # noqa: E731
        w, ws, P, rows, cols, x, xs, P, xss, n, P, kind, ys, None, None)
    assert product(n=0) == product(rows=0) == afx.AFX_OK
    for bad in ({"kind": 3}, {"cols": 0}, {"rows": 1 << 24}, {"n": 1 << 24}, {"cols": 1 << 24}, {"ws": 136}, {"xs": 136}, {"ws": 112}, {"xs": 112},
                {"ws": 1 << 32}, {"ys": 1}, {"cols": 256, "ws": 256, "xs": 256, "xss": 1}, {"w": None}, {"w": P + 8}, {}):
        assert product(**bad) == E


def test_rotary_plans(afx):
    for bad in ({"head_dim": 0}, {"head_dim": 63}, {"head_dim": 258}, {"rotary_dim": 0}, {"rotary_dim": 66}, {"rotary_dim": 3}, {"base": 0.0},
                {"base": math.inf}, {"amplitude": math.nan}, {"base": -1.0}):
        with pytest.raises((afx.AfxError, ValueError)):
            afx.rotary(**{"head_dim": 64, **bad})
    for bad in ({"sections": [16, 15]}, {"sections": []}, {"order": "other"}, {"pairs": "other"}, {"frequencies": [1.0]}, {"sections": [33, -1]},
                {"frequencies": [math.inf] * 32}, {"sections": [4] * 8 + [0]}):
        with pytest.raises((afx.AfxError, ValueError)):
            afx.rotary(64, **bad)
    plan = afx.rotary(64, rotary_dim=16, sections=[2, 3, 3], order="interleaved", base=100.0)
    assert list(plan.axis)[:8] == [0, 1, 2, 0, 1, 2, 1, 2]
    assert (plan.head_dim, plan.rotary_dim, plan.n_axes, plan.amplitude) == (64, 16, 3, 1.0)
    for i in range(8):
        turns = 100.0 ** (-2 * i / 16) / (2 * math.pi)
        assert abs(plan.step[i] / 2.0 ** 64 - turns) <= turns * 2.0 ** -51
    # negative frequencies and more than a turn a position
    plan = afx.rotary(4, frequencies=[-0.25, 7.0])
    assert abs(plan.step[0] / 2.0 ** 64 - (1 - 0.25 / (2 * math.pi))) < 2.0 ** -50
    assert abs(plan.step[1] / 2.0 ** 64 - (7 / (2 * math.pi) - 1)) < 2.0 ** -50
    assert afx._lib.afx_rotary_plan(64, 64, 0, 10.0, None, 1, None, 1.0, None) == afx.AFX_E_ARG


def test_rotation_arguments(afx):
    lib, E = afx._lib, afx.AFX_E_ARG
    plan = afx.rotary(64)
    rotate = lambda p=ctypes.byref(plan), xt=2, yt=2, heads=1, n=2, x=P, y=P + 4096, ts=64, hs=64: lib.afx_rotate(  # noqa: E731
        p, P, n, n, x, xt, 64, 64, heads, y, yt, ts, hs, None)
    assert rotate(n=0) == rotate(heads=0) == afx.AFX_OK
    empty = afx.afx_rotary()
    for bad in ({"p": None}, {"p": ctypes.byref(empty)}, {"xt": 3}, {"yt": 3}, {"heads": 65537}, {"ts": 63}, {"heads": 2, "hs": 32}, {"y": P, "yt": 0}, {}):
        assert rotate(**bad) == E
    cache = afx.afx_kv_cache(P, P, 1024, 64, 64, afx.AFX_FMT_BF16, 4, 16, 1, 64, 0)
    qkv = afx.afx_qkv(P, P, P, 64, 64, 64, 64, 64, 64, 2, 1, 2, 0)
    assert lib.afx_rotate_write(ctypes.byref(plan), P, 2, ctypes.byref(qkv), P, 64, 64, ctypes.byref(cache), P, None, None) == E  # host memory
    assert lib.afx_rotate_write(ctypes.byref(plan), P, 2, None, P, 64, 64, ctypes.byref(cache), P, None, None) == E
    assert lib.afx_rotate_write(ctypes.byref(plan), P, 2, ctypes.byref(qkv), P, 64, 64, None, P, None, None) == E
    with pytest.raises(ValueError):
        afx.afx_rotate(plan, torch.zeros(2, dtype=torch.int32), torch.zeros((2, 1, 64)), torch.zeros((2, 1, 64)))


def test_verify_arguments(afx):
    lib, E = afx._lib, afx.AFX_E_ARG
    size = ctypes.c_uint64(7)
    for n, r in ((0, 0), (4, 16_385), ((1 << 24) + 1, 1)):
        assert lib.afx_verify_workspace(n, r, ctypes.byref(size)) == E and size.value == 7
    assert lib.afx_verify_workspace(10, 2, None) == E
    assert afx.afx_verify_workspace(1000, 3) >= 64_000
    none = afx.afx_sampling(None, None, None, None)

    def verify(logits=P, draft=P, stride=8, kind=2, draft_kind=2, vocab=8, requests=1, n=2, starts=P, workspace=P):
        a = afx.afx_verify_args(logits, draft, stride, stride, kind, draft_kind, vocab, requests, n, 0, starts, P, none, none, P, P)
        return lib.afx_verify(ctypes.byref(a), P, P, None, workspace, 1 << 20, None, None)

    assert lib.afx_verify(None, P, P, None, P, 1 << 20, None, None) == E
    for bad in ({"kind": 3}, {"draft_kind": 3}, {"vocab": 0}, {"vocab": 524_289}, {"requests": 0}, {"requests": 16_385}, {"n": (1 << 24) + 1}, {"stride": 7},
                {"starts": None}, {"logits": None}, {"workspace": None}, {}):  # the last: host memory
        assert verify(**bad) == E


def test_rounding_s_reference():
    """The tests' own rounding to E4M3 against torch's conversion."""
    x = torch.cat([torch.linspace(-448, 448, 4001), torch.exp2(torch.linspace(-14, 8.8, 999)), torch.tensor(ref.e4m3_values()[:127]).float()])
    x = torch.cat([x, torch.full((-len(x) % 127,), 0.0)]).view(-1, 127)
    x = torch.cat([x, torch.full((x.shape[0], 1), 448.0)], 1)
    values, scales = ref.quantize(x.numpy())
    assert (scales == 1).all()
    assert np.array_equal(values, x.to(torch.float8_e4m3fn).double().numpy())


def test_structures_have_the_header_s_layout(afx, tmp_path):
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("gcc not available")
    names = ["afx_rotary", "afx_qkv", "afx_sampling", "afx_verify_args"]
    fields = [(s, f) for s in names for f, _ in getattr(afx, s)._fields_]
    lines = ['#include "afx.h"', "#include <stddef.h>", "#include <stdio.h>", "int main(void) {"]
    lines += [f'printf("%zu\\n", sizeof({s}));' for s in names] + [f'printf("%zu\\n", offsetof({s}, {f}));' for s, f in fields]
    lines += ['printf("%d %d %d %d %d %d %d\\n", AFX_FP8_BLOCK, AFX_TYPE_BF16, AFX_TYPE_FP16, AFX_TYPE_F32, AFX_ROTARY_MAX_PAIRS, '
              "AFX_ROTARY_MAX_AXES, AFX_ROTARY_NEIGHBOURS);", "return 0; }"]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines))
    exe = str(tmp_path / "layout")
    subprocess.run([gcc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()
    want = [ctypes.sizeof(getattr(afx, s)) for s in names] + [getattr(getattr(afx, s), f).offset for s, f in fields]
    want += [afx.AFX_FP8_BLOCK, afx.AFX_TYPE_BF16, afx.AFX_TYPE_FP16, afx.AFX_TYPE_F32, afx.AFX_ROTARY_MAX_PAIRS, afx.AFX_ROTARY_MAX_AXES,
             afx.AFX_ROTARY_NEIGHBOURS]
    assert [int(v) for v in got] == want
