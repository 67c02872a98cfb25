"""The Python binding of the row operators.  Without a device every call here is refused, by the
binding or by the library's own checks, before a launch."""
import pytest
import torch

import bulk_fills_amd as tk

A, B, D, E, F, H = (0x1000000 * k for k in range(1, 7))  # device addresses never dereferenced


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_a_workspace_may_be_an_address(t):
    """Like every other buffer; it then has the bytes that tk_backward_workspace_bytes names, so the
    library looks at its address: misaligned, or inside another argument, it is refused."""
    add, norm, both = (getattr(tk, f"tk_{n}_{t}") for n in ("dropout_add_backward", "layer_norm_backward",
                                                            "dropout_add_layer_norm_backward"))
    for ws in ((1 << 40) + 2, A, A + 64):
        for call in (lambda: add(1, 0, 4000, 8, 0.1, 0, A, None, B, None, H, ws, 0),
                     lambda: norm(4000, 8, 0, A, None, B, None, None, D, E, F, None, H, None, ws, 0),
                     lambda: both(1, 0, 4000, 8, 0.1, 0, A, None, None, None, B, None, None, D, E, F, None, None, None, H, None,
                                  None, ws, 0)):
            with pytest.raises(tk.TkError) as e:
                call()
            assert e.value.code == tk.TK_EINVAL


class OtherStream:
    """A stream of another device than the current one."""
    device_index, cuda_stream = 7, 0


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(tk, "_device", lambda: 0)
    s = OtherStream()
    for t in ("f32", "f16", "bf16"):
        f = lambda n: getattr(tk, f"tk_{n}_{t}")  # noqa: E731
        for call in (lambda: f("dropout_add")(1, 0, 4, 8, 0.1, 0, A, None, None, None, None, B, None, s),
                     lambda: f("dropout_add_backward")(1, 0, 4, 8, 0.1, 0, A, None, B, None, None, None, s),
                     lambda: f("dropout_add_backward")(1, 0, 4000, 8, 0.1, 0, A, None, B, None, H, None, s),
                     lambda: f("layer_norm")(4, 8, 1e-5, 0, A, None, None, None, B, None, None, None, s),
                     lambda: f("layer_norm_backward")(4, 8, 0, A, None, B, None, None, D, E, F, None, None, None, None, s),
                     lambda: f("dropout_add_layer_norm")(1, 0, 4, 8, 0.1, 1e-5, 0, A, None, None, None, None, None, None, None,
                                                         None, B, None, None, None, s),
                     lambda: f("dropout_add_layer_norm_backward")(1, 0, 4, 8, 0.1, 0, A, None, None, None, B, None, None, D, E,
                                                                  F, None, None, None, None, None, None, None, s)):
            with pytest.raises(ValueError, match="stream"):
                call()


@pytest.mark.gpu
def test_an_address_of_a_workspace_serves():
    rows, cols = 3000, 200
    dy, x = torch.randn(rows, cols, device="cuda"), torch.randn(rows, cols, device="cuda")
    mean, rstd = x.mean(1), x.var(1).rsqrt()
    ws = torch.empty(tk.tk_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    out = []
    for w in (None, ws, ws.data_ptr(), (ws.data_ptr(), ws.numel())):
        dx, dg = torch.empty_like(x), torch.empty(cols, device="cuda")
        tk.tk_layer_norm_backward_f32(rows, cols, 0, dy, None, x, None, None, mean, rstd, dx, None, dg, None, w)
        out.append((dx, dg))
    assert all(torch.equal(a, b) for o in out[1:] for a, b in zip(out[0], o))
