"""Argument checks and workspace queries of the gated layers, log probabilities
and distillation, which need no GPU: every malformed call is refused before a
device is looked for (a call that passes all checks ends with FC_E_HIP or
FC_E_UNSUPPORTED here)."""
from __future__ import annotations

import ctypes
import os

import pytest

from sharded_fc_layer_amd import fcshard as F
from test_fused_cpu import SIZES, _changed, at

BAD = F.FC_E_INVALID
T_BAD = (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -11, 2.0 ** 11)
TOP = 128


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(F.LIB_PATH):
        from sharded_fc_layer_amd import build
        build.build()
    return F.lib()


def calls(L):
    """name -> (function, arguments of a call that is right, pointers that must be there, {position: values that
    must be refused}, outputs, inputs)"""
    ws, n = at(20), 1 << 40
    return {
        "fc_fwd_glu": (L.fc_fwd_glu, [at(0), at(1), 0, at(2), 4, at(3), at(4), 0, 8001, 1001, 4003, ws, n, None],
                       (0, 1, 6), {2: (2, -1), 4: (-1, 5), 7: (-1, 2, 3), 8: SIZES, 9: SIZES, 10: SIZES},
                       (5, 6, 11), (0, 1, 3)),
        "fc_bwd_data_glu": (L.fc_bwd_data_glu, [at(0), at(1), 0, at(2), 4, at(3), at(4), at(5), 8001, 4003, 1001, ws, n,
                                                None],
                            (0, 1, 3, 5), {2: (2, -1), 4: (-1, 5), 8: SIZES, 9: SIZES, 10: SIZES}, (5, 6, 7, 11),
                            (0, 1, 3)),
        "fc_bwd_glu": (L.fc_bwd_glu, [at(0), at(1), 4, at(2), at(3), at(4), 65, 33, ws, n, None],
                       (0, 1), {2: (-1, 5), 6: SIZES, 7: SIZES}, (3, 4, 5, 8), (0, 1)),
        "fc_logprob": (L.fc_logprob, [at(0), at(1), 0, at(2), 0, -100, 1.0, at(3), at(4), at(5), at(6), at(7), 20, 8001,
                                      1001, 8003, ws, n, None],
                       (0, 1, 3, 7, 9, 10, 11), {2: (2, -1), 4: (-1,), 6: T_BAD, 12: (-1, TOP + 1), 13: SIZES,
                                                 14: SIZES, 15: SIZES}, (7, 8, 9, 10, 11, 16), (0, 1, 3)),
        "fc_distill_fwd": (L.fc_distill_fwd, [at(0), at(1), 0, at(2), at(3), 20, 0, 2.0, at(4), at(5), at(6), 8001, 1001,
                                              8003, ws, n, None],
                           (0, 1, 3, 4, 8, 9, 10), {2: (2, -1), 5: (0, -1, TOP + 1), 6: (-1,), 7: T_BAD, 11: SIZES,
                                                    12: SIZES, 13: SIZES}, (8, 9, 10, 14), (0, 1, 3, 4)),
        "fc_distill_bwd": (L.fc_distill_bwd, [at(0), at(1), 0, at(2), at(3), 20, 0, 2.0, at(4), at(5), at(6), at(7), 0,
                                              at(8), 0, 8001, 1001, 8003, ws, n, None],
                           (0, 1, 3, 4, 8, 9, 10, 11, 13), {2: (2, -1), 5: (0, -1, TOP + 1), 6: (-1,), 7: T_BAD,
                                                            12: (-1, 2, 3), 14: (-1, 3), 15: SIZES, 16: SIZES,
                                                            17: SIZES}, (11, 13, 18), (0, 1, 3, 4, 8, 9, 10)),
    }


NAMES = ("fc_fwd_glu", "fc_bwd_data_glu", "fc_bwd_glu", "fc_logprob", "fc_distill_fwd", "fc_distill_bwd")


@pytest.mark.parametrize("name", NAMES)
def test_malformed_arguments_are_refused(L, name):
    import torch
    fn, args, needed, wrong, _, _ = calls(L)[name]
    if not torch.cuda.is_available():  # the addresses are made up: with a device the call would run
        assert fn(*args) in (F.FC_E_HIP, F.FC_E_UNSUPPORTED)
    for p in needed:
        assert fn(*_changed(args, p, None)) == BAD, f"NULL argument {p}"
    for p, values in wrong.items():
        for v in values:
            assert fn(*_changed(args, p, v)) == BAD, f"argument {p} = {v}"
    pointers = [p for p, a in enumerate(args) if isinstance(a, ctypes.c_void_p)]
    for p in pointers:  # odd addresses
        assert fn(*_changed(args, p, ctypes.c_void_p(args[p].value + 1))) == BAD, f"odd address of argument {p}"
    w = pointers[-1]  # the workspace: missing, too small, misaligned
    for v in (None, ctypes.c_void_p(args[w].value + 16)):
        assert fn(*_changed(args, w, v)) == BAD
    assert fn(*_changed(args, w + 1, 0)) == BAD


@pytest.mark.parametrize("name", NAMES)
def test_overlapping_outputs_are_refused(L, name):
    fn, args, _, _, outs, ins = calls(L)[name]
    for o in outs:
        for i in ins + tuple(p for p in outs if p != o):
            assert fn(*_changed(args, o, args[i])) == BAD, f"output {o} on argument {i}"


def test_what_may_be_missing(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")

    def without(name, *positions):
        fn, args = calls(L)[name][:2]
        for p in positions:
            args = _changed(args, p, 0 if isinstance(args[p], int) else None)
        return fn(*args)

    assert without("fc_fwd_glu", 3, 5) != BAD
    assert without("fc_bwd_data_glu", 6, 7) != BAD
    assert without("fc_bwd_glu", 3, 4) != BAD and without("fc_bwd_glu", 4, 5, 8, 9) != BAD
    assert without("fc_bwd_glu", 3, 4, 5) == BAD  # no output
    assert without("fc_logprob", 3, 7) != BAD and without("fc_logprob", 8) != BAD
    assert without("fc_logprob", 10, 11, 12) != BAD  # no alternatives
    fn, args = calls(L)["fc_logprob"][:2]
    assert fn(*_changed(_changed(args, 15, 19), 12, 20)) == BAD  # more alternatives than columns


def test_a_call_takes_what_its_query_says(L):
    """One byte less than the query's answer is refused, the answer itself is not."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    queries = {"fc_fwd_glu": lambda: L.fc_fwd_glu_ws_bytes(333, 1001, 403, 0, 1),
               "fc_bwd_data_glu": lambda: L.fc_bwd_data_glu_ws_bytes(8001, 4003, 1001, 0, 1),
               "fc_bwd_glu": lambda: L.fc_bwd_glu_ws_bytes(65, 33),
               "fc_logprob": lambda: L.fc_logprob_ws_bytes(8001, 1001, 8003, 0, 20, 1),
               "fc_distill_fwd": lambda: L.fc_distill_fwd_ws_bytes(8001, 1001, 8003, 0, 1),
               "fc_distill_bwd": lambda: L.fc_distill_bwd_ws_bytes(8001, 1001, 8003, 0, 20, 1)}
    for name, query in queries.items():
        fn, args = calls(L)[name][:2]
        if name == "fc_fwd_glu":
            args = args[:8] + [333, 1001, 403] + args[11:]
        need, w = query(), [p for p, a in enumerate(args) if isinstance(a, ctypes.c_void_p)][-1]
        assert need > 0 and need % 256 == 0
        assert fn(*_changed(args, w + 1, need - 1)) == BAD, name
        assert fn(*_changed(args, w + 1, need)) != BAD, name


def test_workspace_queries(L):
    for bad in SIZES:
        for dims in ((bad, 8, 8), (8, bad, 8), (8, 8, bad)):
            assert L.fc_fwd_glu_ws_bytes(*dims, 0, 1) == -1
            assert L.fc_bwd_data_glu_ws_bytes(*dims, 0, 1) == -1
            assert L.fc_logprob_ws_bytes(*dims, 0, 1, 1) == -1
            assert L.fc_distill_fwd_ws_bytes(*dims, 0, 1) == -1
            assert L.fc_distill_bwd_ws_bytes(*dims, 0, 1, 1) == -1
        assert L.fc_bwd_glu_ws_bytes(bad, 8) == -1 and L.fc_bwd_glu_ws_bytes(8, bad) == -1
    for k in (-1, 9, TOP + 1):
        assert L.fc_logprob_ws_bytes(8, 8, 8, 0, k, 1) == -1
    for n in (-1, 0, TOP + 1):
        assert L.fc_distill_bwd_ws_bytes(8, 8, 8, 0, n, 1) == -1
    assert L.fc_fwd_glu_ws_bytes(8, 8, 8, 2, 1) == -1 and L.fc_logprob_ws_bytes(8, 8, 8, -1, 1, 1) == -1
    # logits are held for some rows at a time, not whole
    M, K, N = 8192, 2048, 128256
    for need in (L.fc_logprob_ws_bytes(M, K, N, 0, 20, 1), L.fc_distill_fwd_ws_bytes(M, K, N, 0, 1)):
        assert 1 << 29 < need < M * N * 4 // 3
    assert L.fc_logprob_ws_bytes(M, K, N, 0, 0, 1) < 1 << 28  # statistics alone
    # no query overflows at the largest sizes
    top = 1 << 22
    for q in (L.fc_fwd_glu_ws_bytes(top, top, top, 0, 0), L.fc_bwd_data_glu_ws_bytes(top, top, top, 0, 0),
              L.fc_logprob_ws_bytes(top, top, top, 0, 128, 0), L.fc_distill_fwd_ws_bytes(top, top, top, 0, 0),
              L.fc_distill_bwd_ws_bytes(top, top, top, 0, 128, 0)):
        assert q > 0


def test_binding_refuses_what_is_not_on_the_gpu():
    import torch
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    w = torch.zeros(8, 16, dtype=torch.bfloat16)
    for call in (lambda: F.fc_fwd_glu(x, w), lambda: F.fc_bwd_glu(x, w), lambda: F.fc_logprob(x, w),
                 lambda: F.fc_distill_fwd(x, w, torch.zeros(4, 1, dtype=torch.int64), torch.zeros(4, 1))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
