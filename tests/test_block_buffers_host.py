"""Blobs, workspaces and status words of another type, layout or size are refused by the binding (no GPU needed).  The
operands pass as ones on GPU 0; the library's calls only note that they were reached."""
import pytest
import torch

from mixed_precision_decode_b200 import build

build.build()

from mixed_precision_decode_b200 import bitsmoe as B  # noqa: E402

E, K, D, F, T, G = 4, 2, 16, 32, 6, 32


@pytest.fixture
def reached(monkeypatch):
    calls = []
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(B, "_launch", lambda what, *a: calls.append(what))
    return calls


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _u8(n):
    return torch.zeros(n, dtype=torch.uint8)


def _calls(name, **kw):
    """The operator with good operands and kw in the place of some of them."""
    d = B.ffn_dims(D, F, E, K)
    W, W2, x = torch.zeros(E, F, D).half(), torch.zeros(E, D, F).half(), torch.zeros(T, D).half()
    y, gw, ids = torch.zeros(T, K, F), torch.zeros(T, K), _i32(T, K)
    blob = kw.pop("blob", _u8(B.q4_bytes(E, D, F, G)))
    n = kw.pop("workspace_bytes", 1024)
    ws = kw.pop("workspace", _u8(n))
    if name == "topk_route":
        B.topk_route(torch.zeros(T, E), ids, gw, workspace=ws, **kw)
    elif name == "q4_pack":
        B.q4_pack(W2, G, blob, **kw)
    elif name == "q4_unpack":
        B.q4_unpack(blob, G, W2.float(), **kw)
    elif name == "ffn_down_q4":
        B.ffn_down_q4(d, blob, G, y, y, ids, gw, T, torch.zeros(T, D), ws, n, **kw)
    elif name == "grouped_matmul":
        B.grouped_matmul(x, W, _i32(E + 1), torch.zeros(T, F), **kw)
    else:
        B.dense_ffn_forward(d, W, W, W2, x, ids, gw, _i32(E + 1), _i32(T * K), torch.zeros(T, D), ws, **kw)


ALL = ("topk_route", "q4_pack", "q4_unpack", "ffn_down_q4", "grouped_matmul", "dense_ffn_forward")


def _code(name, **kw):
    with pytest.raises(B.BitsMoEError) as e:
        _calls(name, **kw)
    return e.value.code


@pytest.mark.parametrize("name", ALL)
def test_good_buffers_pass(reached, name):
    _calls(name)
    if name != "q4_unpack":
        _calls(name, status=_i32(1))
    assert set(reached) == {name}


@pytest.mark.parametrize("name", [n for n in ALL if n != "q4_unpack"])
@pytest.mark.parametrize("status", [torch.zeros(1), torch.zeros(1, dtype=torch.int64), _u8(4), _i32(0)])
def test_status_of_another_type(reached, name, status):
    assert _code(name, status=status) == B.EINVAL and not reached


@pytest.mark.parametrize("name", ["q4_pack", "q4_unpack", "ffn_down_q4"])
def test_blob_of_another_type_layout_or_size(reached, name):
    n = B.q4_bytes(E, D, F, G)
    assert _code(name, blob=_u8(2 * n)[::2]) == B.EINVAL
    assert _code(name, blob=torch.zeros(n, dtype=torch.int8)) == B.EINVAL
    assert _code(name, blob=torch.zeros(n // 4, dtype=torch.float32)) == B.EINVAL
    assert _code(name, blob=_u8(n - 1)) == B.ESIZE
    assert not reached


@pytest.mark.parametrize("name", ["topk_route", "ffn_down_q4", "dense_ffn_forward"])
def test_workspace_with_gaps(reached, name):
    assert _code(name, workspace=_u8(2048)[::2], workspace_bytes=1024) == B.EINVAL and not reached


def test_workspace_smaller_than_said(reached):
    """The kernels go by workspace_bytes: it must not be more than the tensor holds."""
    assert _code("ffn_down_q4", workspace=_u8(1023), workspace_bytes=1024) == B.ESIZE and not reached
    _calls("ffn_down_q4", workspace=_u8(1025), workspace_bytes=1024)
    _calls("ffn_down_q4", workspace=None, workspace_bytes=0)
