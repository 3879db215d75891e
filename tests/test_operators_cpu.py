"""The operators at the ends of the model without a GPU: sizes of workspaces and
every refusal, before anything reaches a device."""
import ctypes

import pytest
import torch

from recurrent_memory_transformer_diag_b200 import armt, operators as ops
from recurrent_memory_transformer_diag_b200.armt import ArmtError

OK, INVALID, UNSUPPORTED = 0, 1, 7
A = 1 << 20   # a well-aligned address that nothing reads


def size(lib, name, *args):
    n = ctypes.c_size_t(99)
    return getattr(lib, name)(*args, ctypes.byref(n)), n.value


def test_workspace_sizes(libarmt):
    assert size(libarmt, "armt_embed_grad_workspace", 1, 128, 1000, 64) == (OK, 0)
    s, n = size(libarmt, "armt_embed_grad_workspace", 1, 129, 1000, 64)
    assert s == OK and n > 129 * 16
    s, a = size(libarmt, "armt_token_loss_workspace", 1, 1 << 17, 1 << 17, 2048, 0)
    s2, b = size(libarmt, "armt_token_loss_workspace", 1, 8192, 1 << 17, 2048, 0)
    assert (s, s2) == (OK, OK) and a == b < 1 << 28     # rows come in passes
    s, g = size(libarmt, "armt_token_loss_workspace", 1, 8192, 1 << 17, 2048, 1)
    assert s == OK and g < 1 << 30                      # the logits alone would take 2 GiB and more
    s, n = size(libarmt, "armt_rms_norm_grad_workspace", 1, 1, 64)
    assert (s, n) == (OK, 64 * 4)


@pytest.mark.parametrize("name,args,status", [
    ("armt_embed_grad_workspace", (1, 0, 8, 64), INVALID), ("armt_embed_grad_workspace", (1, 8, 0, 64), INVALID),
    ("armt_embed_grad_workspace", (2, 8, 8, 64), INVALID), ("armt_embed_grad_workspace", (1, 8, 8, 60), UNSUPPORTED),
    ("armt_rms_norm_grad_workspace", (1, 8, 16392), UNSUPPORTED), ("armt_rms_norm_grad_workspace", (3, 8, 64), INVALID),
    ("armt_embed_grad_workspace", (1, (1 << 30) + 1, 8, 64), UNSUPPORTED),
    ("armt_token_loss_workspace", (1, 8, (1 << 30) + 1, 64, 0), UNSUPPORTED),
    ("armt_token_loss_workspace", (1, 8, 8, (1 << 20) + 8, 0), UNSUPPORTED),
    ("armt_rms_norm_grad_workspace", (0, 8, -8), INVALID), ("armt_token_loss_workspace", (1, -1, 8, 64, 0), INVALID),
    ("armt_token_loss_workspace", (1, 8, 8, 64, 2), INVALID), ("armt_token_loss_workspace", (0, 8, 8, 4, 1), UNSUPPORTED),
])
def test_workspace_refusals(libarmt, name, args, status):
    assert size(libarmt, name, *args) == (status, 0)


EMBED = dict(dtype=1, n=4, vocab=8, d=64, ids=A, id_bytes=8, table=A, scale=1.0, out=A, stream=None)
EMBED_GRAD = dict(dtype=1, n=4, vocab=8, d=64, ids=A, id_bytes=8, d_out=A, scale=1.0, d_table=A, accumulate=0,
                  workspace=None, bytes=0, stream=None)
NORM = dict(dtype=1, n=4, d=64, x=A, gain=A, eps=1e-5, y=A, rstd=None, stream=None)
NORM_GRAD = dict(dtype=1, n=4, d=64, x=A, gain=A, rstd=A, dy=A, dx=A, d_gain=A, workspace=A, bytes=1 << 30, stream=None)
LOSS = dict(dtype=1, n=4, vocab=8, d=64, hidden=A, head=A, targets=A, target_bytes=8, scale=1.0, loss=A, lse=A,
            workspace=A, bytes=1 << 40, stream=None)
LOSS_GRAD = dict(dtype=1, n=4, vocab=8, d=64, hidden=A, head=A, targets=A, target_bytes=8, scale=1.0, lse=A, d_loss=A,
                 d_hidden=A, d_head=A, workspace=A, bytes=1 << 40, stream=None)
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("name,base,change,status", [
    (f, b, c, s) for f, b, changes in [
        ("armt_embed", EMBED, [dict(n=0), dict(vocab=-1), dict(ids=None), dict(table=None), dict(out=None),
                               dict(id_bytes=2), dict(scale=NAN), dict(table=A + 2), dict(out=A + 8), dict(dtype=2)]),
        ("armt_embed_grad", EMBED_GRAD, [dict(n=0), dict(ids=None), dict(d_out=None), dict(d_table=None),
                                         dict(id_bytes=0), dict(scale=INF), dict(accumulate=2), dict(d_out=A + 4),
                                         dict(n=5000), dict(n=5000, workspace=A, bytes=100),
                                         dict(n=5000, workspace=A + 8, bytes=1 << 30)]),
        ("armt_rms_norm", NORM, [dict(d=0), dict(x=None), dict(gain=None), dict(y=None), dict(eps=-1.0), dict(eps=NAN),
                                 dict(x=A + 2), dict(gain=A + 4), dict(dtype=3)]),
        ("armt_rms_norm_grad", NORM_GRAD, [dict(x=None), dict(gain=None), dict(rstd=None), dict(dy=None), dict(dx=None),
                                           dict(d_gain=None), dict(workspace=None), dict(bytes=1), dict(dx=A + 2)]),
        ("armt_token_loss", LOSS, [dict(n=0), dict(vocab=0), dict(hidden=None), dict(head=None), dict(targets=None),
                                   dict(loss=None), dict(lse=None), dict(workspace=None), dict(bytes=512),
                                   dict(target_bytes=1), dict(scale=INF), dict(head=A + 8), dict(dtype=2)]),
        ("armt_token_loss_grad", LOSS_GRAD, [dict(lse=None), dict(d_loss=None), dict(d_hidden=None, d_head=None),
                                             dict(workspace=None), dict(bytes=0), dict(scale=NAN), dict(d_head=A + 4),
                                             dict(d_hidden=A + 2), dict(target_bytes=16), dict(targets=None)]),
    ] for c, s in [(c, INVALID) for c in changes] + [(dict(d=60), UNSUPPORTED)]
] + [("armt_rms_norm", NORM, dict(d=16392), UNSUPPORTED)])
def test_refusals(libarmt, name, base, change, status):
    args = {**base, **change}
    assert getattr(libarmt, name)(*args.values()) == status


def test_status_of_no_workspace(libarmt):
    assert libarmt.armt_workspace_status(None, None) == INVALID
    assert libarmt.armt_test_loss_wait(0, None) == INVALID


def test_wrappers_refuse_tensors_off_the_device():
    x = torch.zeros(4, 64)
    i = torch.zeros(4, dtype=torch.int64)
    v = torch.zeros(4)
    for call in (lambda: ops.embed(i, x, x.clone()), lambda: ops.embed_grad(i, x, x.clone()),
                 lambda: ops.rms_norm(x, x[0], x.clone()), lambda: ops.rms_norm_grad(x, x[0], v, x, x, x[0]),
                 lambda: ops.token_loss(x, x, i, v, v), lambda: ops.token_loss_grad(x, x, i, v, v, x, x)):
        with pytest.raises(ArmtError, match="CUDA device") as e:
            call()
        assert e.value.status == INVALID


def test_workspace_bytes(libarmt):
    assert ops.workspace_bytes("embed_grad", torch.bfloat16, 10, 64, 100) == 0
    assert ops.workspace_bytes("token_loss", torch.float32, 10, 64, 100) > \
        ops.workspace_bytes("token_loss", torch.bfloat16, 10, 64, 100) > 0
    with pytest.raises(ArmtError):
        ops.workspace_bytes("token_loss", torch.float16, 10, 64, 100)
    with pytest.raises(ArmtError):
        ops.workspace_bytes("loss", torch.float32, 10, 64, 100)
    with pytest.raises(ArmtError) as e:
        ops.workspace_bytes("rms_norm_grad", torch.float32, 10, 60)
    assert e.value.status == UNSUPPORTED


def test_exports_are_bound(libarmt):
    for name in ("armt_embed", "armt_rms_norm", "armt_token_loss", "armt_token_loss_grad", "armt_workspace_status"):
        assert name in armt.EXPORTS and getattr(libarmt, name).argtypes


@pytest.mark.parametrize("name,base,change", [
    (f, b, c) for f, b, changes in [
        ("armt_embed", EMBED, [dict(ids=A + 4), dict(ids=A + 2, id_bytes=4)]),
        ("armt_embed_grad", EMBED_GRAD, [dict(ids=A + 4), dict(ids=A + 1, id_bytes=4)]),
        ("armt_rms_norm", NORM, [dict(rstd=A + 2)]),
        ("armt_rms_norm_grad", NORM_GRAD, [dict(rstd=A + 2), dict(d_gain=A + 1), dict(d_gain=A + 2, dtype=0)]),
        ("armt_token_loss", LOSS, [dict(targets=A + 4), dict(targets=A + 3, target_bytes=4), dict(loss=A + 2),
                                   dict(lse=A + 1)]),
        ("armt_token_loss_grad", LOSS_GRAD, [dict(targets=A + 4), dict(lse=A + 2), dict(d_loss=A + 3)]),
    ] for c in changes])
def test_refusals_of_numbers_off_their_own_size(libarmt, name, base, change):
    """ids, targets and single numbers a row need no 16-byte boundary, but their own size."""
    assert getattr(libarmt, name)(*{**base, **change}.values()) == INVALID


@pytest.mark.parametrize("workspace", [None, 5, torch.zeros(64, dtype=torch.uint8)])
def test_status_of_what_is_no_workspace(workspace):
    with pytest.raises(ArmtError, match="CUDA device") as e:
        ops.workspace_status(workspace)
    assert e.value.status == INVALID
