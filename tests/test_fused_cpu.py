"""The fused operators' argument checks and workspace queries, which need no
GPU: every malformed call is refused before a device is looked for (a call
that passes all checks ends with FC_E_HIP or FC_E_UNSUPPORTED here)."""
from __future__ import annotations

import ctypes
import os

import pytest

from sharded_fc_layer_amd import fcshard as F

BAD = F.FC_E_INVALID


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(F.LIB_PATH):
        from sharded_fc_layer_amd import build
        build.build()
    return F.lib()


def at(i):
    """Addresses far apart, aligned, never touched: the checks read no memory."""
    return ctypes.c_void_p(0x100000000 * (i + 1))


# name -> (arguments of a call that is right, positions of pointers that must
# be there, {position: values that must be refused})
SIZES = (0, -1, (1 << 22) + 1, -(1 << 63))


def calls(L):
    ws, n = at(20), 1 << 40
    d3 = {p: SIZES for p in (10, 11, 12)}
    return {
        "fc_fwd_act": (L.fc_fwd_act, [at(0), 0, at(1), 0, at(2), at(3), 3, at(4), at(5), 0, 8001, 1001, 8003, ws, n, None],
                       (0, 2, 8), {1: (2, -1), 3: (2, -1), 6: (-1, 5), 9: (-1, 2, 3), **d3}),
        "fc_bwd_data_act": (L.fc_bwd_data_act, [at(0), at(1), 0, at(2), 1, at(3), 0, at(4), 8001, 8003, 1001, ws, n, None],
                            (0, 1, 3, 5), {2: (2, -1), 4: (-1, 5), 6: (-1, 2, 3), 8: SIZES, 9: SIZES, 10: SIZES}),
        "fc_bwd_act": (L.fc_bwd_act, [at(0), at(1), 2, at(2), at(3), 65, 33, ws, n, None],
                       (0, 1), {2: (-1, 5), 5: SIZES, 6: SIZES}),
        "fc_xent_fwd": (L.fc_xent_fwd, [at(0), at(1), 0, at(2), 0, -100, at(3), at(4), at(5), 8001, 1001, 8003, ws, n, None],
                        (0, 1, 3, 6, 7), {2: (2, -1), 4: (-1,), 9: SIZES, 10: SIZES, 11: SIZES}),
        "fc_xent_bwd": (L.fc_xent_bwd, [at(0), at(1), 0, at(2), 0, -100, at(3), at(4), at(5), 0, at(6), 0, 8001, 1001, 8003,
                                        ws, n, None],
                        (0, 1, 3, 6, 7, 8, 10), {2: (2, -1), 4: (-1,), 9: (-1, 2, 3), 11: (-1, 3), 12: SIZES,
                                                 13: SIZES, 14: SIZES}),
        "fc_grouped_fwd": (L.fc_grouped_fwd, [at(0), at(1), 0, at(2), at(3), 0, 30001, 3, 2603, 2605, ws, n, None],
                           (0, 1, 3, 4), {2: (2, -1), 5: (-1, 2, 3), 6: SIZES, 7: (0, -1, (1 << 20) + 1), 8: SIZES,
                                          9: SIZES}),
        "fc_grouped_bwd_data": (L.fc_grouped_bwd_data, [at(0), at(1), 1, at(2), at(3), 1, 30001, 3, 2603, 2605, ws, n, None],
                                (0, 1, 3, 4), {2: (2, -1), 5: (-1, 2, 3), 6: SIZES, 7: (0, -1, (1 << 20) + 1),
                                               8: SIZES, 9: SIZES}),
        "fc_grouped_bwd_weight": (L.fc_grouped_bwd_weight, [at(0), at(1), at(2), at(3), 2, 30001, 3, 2603, 2605, ws, n, None],
                                  (0, 1, 2, 3), {4: (-1, 3), 5: SIZES, 6: (0, -1, (1 << 20) + 1), 7: SIZES,
                                                 8: SIZES}),
    }


NAMES = ("fc_fwd_act", "fc_bwd_data_act", "fc_bwd_act", "fc_xent_fwd", "fc_xent_bwd", "fc_grouped_fwd",
         "fc_grouped_bwd_data", "fc_grouped_bwd_weight")


def _changed(args, p, v):
    out = list(args)
    out[p] = v
    return out


@pytest.mark.parametrize("name", NAMES)
def test_malformed_arguments_are_refused(L, name):
    import torch
    fn, args, needed, wrong = calls(L)[name]
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


@pytest.mark.parametrize("name, outs, ins", [
    ("fc_fwd_act", (7, 8, 13), (0, 2, 4, 5)), ("fc_bwd_data_act", (5, 7, 11), (0, 1, 3)),
    ("fc_bwd_act", (3, 4, 7), (0, 1)), ("fc_xent_fwd", (6, 7, 8, 12), (0, 1, 3)),
    ("fc_xent_bwd", (8, 10, 15), (0, 1, 3, 6, 7)), ("fc_grouped_fwd", (4, 10), (0, 1, 3)),
    ("fc_grouped_bwd_data", (4, 10), (0, 1, 3)), ("fc_grouped_bwd_weight", (3, 9), (0, 1, 2))])
def test_overlapping_outputs_are_refused(L, name, outs, ins):
    fn, args, _, _ = calls(L)[name]
    for o in outs:
        for i in ins + tuple(p for p in outs if p != o):
            assert fn(*_changed(args, o, args[i])) == BAD, f"output {o} on argument {i}"


def test_an_activation_gradient_needs_its_z_and_an_output(L):
    fn, args, _, _ = calls(L)["fc_bwd_act"]
    none = _changed(args, 2, F.ACT_NONE)
    assert fn(*_changed(_changed(none, 3, None), 4, None)) == BAD  # neither output
    assert fn(*_changed(args, 1, None)) == BAD  # a slope without Z
    if not __import__("torch").cuda.is_available():
        assert fn(*_changed(none, 1, None)) != BAD
        nodb = _changed(_changed(_changed(args, 4, None), 7, None), 8, 0)
        assert fn(*nodb) != BAD  # no workspace without the column sums


def test_a_call_takes_what_its_query_says(L):
    """One byte less than the query's answer is refused, the answer itself is not."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    for name, query in (("fc_fwd_act", lambda: L.fc_fwd_act_ws_bytes(8001, 1001, 8003, 0, 0, 1)),
                        ("fc_bwd_data_act", lambda: L.fc_bwd_data_act_ws_bytes(8001, 8003, 1001, 0, 1)),
                        ("fc_bwd_act", lambda: L.fc_bwd_act_ws_bytes(65, 33)),
                        ("fc_xent_fwd", lambda: L.fc_xent_fwd_ws_bytes(8001, 1001, 8003, 0, 1)),
                        ("fc_xent_bwd", lambda: L.fc_xent_bwd_ws_bytes(8001, 1001, 8003, 0, 1)),
                        ("fc_grouped_fwd", lambda: L.fc_grouped_ws_bytes(0, 30001, 3, 2603, 2605, 0, 1)),
                        ("fc_grouped_bwd_data", lambda: L.fc_grouped_ws_bytes(1, 30001, 3, 2603, 2605, 1, 1)),
                        ("fc_grouped_bwd_weight", lambda: L.fc_grouped_ws_bytes(2, 30001, 3, 2603, 2605, 0, 1))):
        fn, args, _, _ = calls(L)[name]
        need, w = query(), [p for p, a in enumerate(args) if isinstance(a, ctypes.c_void_p)][-1]
        assert need > 0 and need % 256 == 0
        assert fn(*_changed(args, w + 1, need - 1)) == BAD, name
        assert fn(*_changed(args, w + 1, need)) != BAD, name


def test_workspace_queries(L):
    for bad in SIZES:
        for dims in ((bad, 8, 8), (8, bad, 8), (8, 8, bad)):
            assert L.fc_fwd_act_ws_bytes(*dims, 0, 0, 1) == -1
            assert L.fc_bwd_data_act_ws_bytes(*dims, 0, 1) == -1
            assert L.fc_xent_fwd_ws_bytes(*dims, 0, 1) == -1
            assert L.fc_xent_bwd_ws_bytes(*dims, 0, 1) == -1
            assert L.fc_grouped_ws_bytes(0, dims[0], 4, dims[1], dims[2], 0, 1) == -1
        assert L.fc_bwd_act_ws_bytes(bad, 8) == -1 and L.fc_bwd_act_ws_bytes(8, bad) == -1
    assert L.fc_fwd_act_ws_bytes(8, 8, 8, 2, 0, 1) == -1 and L.fc_fwd_act_ws_bytes(8, 8, 8, 0, 2, 1) == -1
    assert L.fc_grouped_ws_bytes(3, 8, 4, 8, 8, 0, 1) == -1 and L.fc_grouped_ws_bytes(0, 8, 0, 8, 8, 0, 1) == -1
    # experts' weights past 2^46 elements
    assert L.fc_grouped_ws_bytes(0, 8, 1 << 20, 1 << 14, 1 << 14, 0, 1) == -1
    # aligned operands of whole rows are read in place
    assert L.fc_fwd_act_ws_bytes(8192, 2048, 8192, 0, 0, 1) == 0
    assert L.fc_grouped_ws_bytes(0, 8192, 8, 2048, 8192, 0, 1) == 0
    # others are copied where the large tiles run: rows of 1001 values padded to 1024
    assert L.fc_grouped_ws_bytes(2, 30000, 8, 1001, 2048, 0, 1) == 30000 * 1024 * 2
    assert L.fc_grouped_ws_bytes(2, 30000, 8, 1024, 2048, 0, 0) == 30000 * (1024 + 2048) * 2
    # the smaller tiles read them where they are
    assert L.fc_fwd_act_ws_bytes(300, 201, 77, 0, 0, 0) == 0
    assert L.fc_fwd_act_ws_bytes(20, 1001, 4099, 0, 1, 0) == 0
    # the gradient of the logits is held a piece at a time, not whole
    M, K, N = 8192, 2048, 128256
    assert L.fc_xent_bwd_ws_bytes(M, K, N, 0, 1) < M * N * 2 // 4 + 4 * M * K
    # no query overflows at the largest sizes
    for q in (L.fc_xent_bwd_ws_bytes, L.fc_xent_fwd_ws_bytes, L.fc_bwd_data_act_ws_bytes):
        assert q(1 << 22, 1 << 22, 1 << 22, 0, 0) > 0


def test_activation_numbers_match_the_header():
    import re
    text = open(F.HEADER).read()
    for name in ("NONE", "RELU", "GELU", "GELU_TANH", "SILU"):
        assert re.search(rf"\bFC_ACT_{name}\s*=\s*{getattr(F, 'ACT_' + name)}\b", text), name


def test_binding_refuses_what_is_not_on_the_gpu():
    import torch
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    w = torch.zeros(8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        F.fc_fwd_act(x, w)
    with pytest.raises(TypeError):
        F.fc_fwd_act(x.float(), w)
    with pytest.raises(ValueError, match="CUDA"):
        F.fc_xent_fwd(x, w, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        F.fc_grouped_fwd(x, w[None], torch.zeros(2, dtype=torch.int64))


# ---- which kernel the planner takes, as the workspaces show it

def up(v, a):
    return -(-v // a) * a


def copied(rows, cols, aligned=True):
    """Bytes of an operand's copy for the 256 x 256 tiles: rows padded to 64 values, none if they fit as they are."""
    return 0 if cols % 8 == 0 and aligned else up(rows * up(cols, 64) * 2, 256)


def weight(K, N, order, aligned=True):
    return copied(K, N, aligned) if order == F.ROW else copied(N, K, aligned)


def test_shapes_of_the_large_tiles_go_there(L):
    """The GPU tests of the 256 x 256 tiles use shapes that the planner sends there. Those leave two rows of
    column sums for 256 rows, two statistics for 256 columns (the 128 x 128 tiles four), planes never, and
    copies where rows do not fit, which the smaller tiles do not make."""
    import test_gpu_fused as G
    for order in (F.ROW, F.COL):
        for M, N, K in G.RING + [(4096, 100, 4096)]:  # fc_bwd_data_act: the reduction is N
            assert L.fc_bwd_data_act_ws_bytes(M, K, N, order, 1) == \
                copied(M, N) + weight(K, N, order) + up(2 * -(-M // 256) * K * 4, 256), (M, N, K)
        for M, K, N in G.RING + [(4100, 640, 1500)]:
            # fc_fwd_act and fc_xent_fwd are planned alike; the statistics show it where nothing is copied
            w = copied(M, K) + weight(K, N, order)
            assert L.fc_xent_fwd_ws_bytes(M, K, N, order, 1) == w + up(2 * 2 * -(-N // 256) * M * 4, 256), (M, K, N)
            assert L.fc_fwd_act_ws_bytes(M, K, N, F.ROW, order, 1) == w
            assert L.fc_fwd_act_ws_bytes(M, K, N, F.COL, order, 1) == copied(K, M) + weight(K, N, order)
        for M, K, N in G.RING_XENT_BWD:
            assert L.fc_xent_bwd_ws_bytes(M, K, N, order, 1) == \
                copied(M, K) + weight(K, N, order) + up(M * up(N, 64) * 2, 256) + 256, (M, K, N)
        for counts, first, behind, K, N in G.RING_GROUPED:
            E, T = len(counts), first + sum(counts) + behind
            for op, A in ((F.OP_FWD, K), (F.OP_BWD_DATA, N), (F.OP_BWD_WEIGHT, K)):
                if K < 1000 and op != F.OP_FWD:
                    continue  # few outputs: not worth the copies
                b = copied(T, N, False) if op == F.OP_BWD_WEIGHT else \
                    copied(E * K, N, False) if order == F.ROW else copied(E * N, K, False)
                assert L.fc_grouped_ws_bytes(op, T, E, K, N, order, 0) == copied(T, A, False) + b, (T, E, K, N, op)
        for M, K, N in G.LAST_PIECE:  # the last piece has 33 columns; the copy shows the large tiles
            piece = (1 << 28) // (2 * M) // 256 * 256
            assert 0 < N % piece < 64 and N > piece
            assert L.fc_xent_bwd_ws_bytes(M, K, N, order, 1) == \
                weight(K, N, order) + up(M * piece * 2, 256) + 256 + M * up(K, 64) * 4
