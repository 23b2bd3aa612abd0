"""Every call of the binding runs with its tensors' device current and on that
device's stream, whatever device the caller has current: a default stream's
handle is 0 on every device and would otherwise be the wrong device's.  On the
CPU, with host tensors that say they are on cuda:1 and a library that records."""
import ctypes

import pytest
import torch

import indirect_expert_matmul_b200 as moe


class OnOne(torch.Tensor):
    """A host tensor that says it is on cuda:1."""
    is_cuda = True
    device = torch.device("cuda", 1)

    def get_device(self):
        return 1


def one(*shape, dtype=torch.float32):
    return _empty(*shape, dtype=dtype).zero_().as_subclass(OnOne)


_empty = torch.empty


@pytest.fixture
def calls(monkeypatch):
    real = moe.lib()
    seen = []
    current = [0]

    class Device:
        def __init__(self, d):
            self.d = d.index if isinstance(d, torch.device) else int(d)

        def __enter__(self):
            self.old, current[0] = current[0], self.d

        def __exit__(self, *a):
            current[0] = self.old

    class Stream:
        def __init__(self, i):
            self.cuda_stream = 1000 + i

    class Library:
        def __getattr__(self, name):
            if name.endswith(("_size", "_size_w", "_string")):
                return getattr(real, name)

            def f(*args):
                s = args[-1]
                seen.append((name, current[0], s.value if isinstance(s, ctypes.c_void_p) else s))
                return moe.OK
            return f

    index = lambda d: d if isinstance(d, int) else current[0] if d is None else d.index
    monkeypatch.setattr(moe, "_L", lambda: Library())
    monkeypatch.setattr(moe, "_raw_stream", lambda i: 1000 + i)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(index(d)))
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: _empty(*a, **kw).as_subclass(OnOne))
    monkeypatch.setattr(torch, "empty_like", lambda t: _empty(t.shape, dtype=t.dtype).as_subclass(OnOne))
    return seen


def test_every_call_runs_on_its_tensors_device(calls):
    u8, i32 = torch.uint8, torch.int32
    E, k, T, n, ff = 4, 2, 3, 64, 32
    ids, w, x, dst = one(T, k, dtype=i32), one(T, k), one(T, n), one(T, k, n)
    Wq = moe.weights_prepare(one(E, ff, n // 32, 34, dtype=u8), E, ff, n)
    Wx = moe.weights_prepare(one(E, ff, n // 32, 17, dtype=u8), E, ff, n, wtype="mxfp4")
    Wd = moe.weights_prepare(one(E, n, ff // 32, 34, dtype=u8), E, n, ff)
    moe.row_ids(ids, E)
    moe.mul_mat_id(Wq, E, ff, n, x, ids)
    moe.mul_mat_id_mx4(Wx, E, ff, n, x, ids)
    moe.ffn(Wq, Wq, Wd, E, n, ff, x, ids)
    moe.ffn_decode_noalloc(Wq, Wq, Wd, E, n, ff, x, ids)
    moe.route(one(T, E), k)
    moe.route_scored(one(T, E), k)
    moe.route_scored_backward(one(T, E), ids, w)
    moe.combine(dst, w)
    moe.combine_backward(x, dst, w)
    moe.mxfp4_quantize(x, with_values=True)
    moe.get_status(moe.workspace(T, k, E, n, device="cuda:1"))
    names = {c[0] for c in calls}
    assert names == {"moe_weights_prepare_w", "moe_row_ids", "moe_mul_mat_id_w", "moe_mul_mat_id_mx4", "moe_ffn_w",
                     "moe_ffn_decode_noalloc", "moe_route", "moe_route_scored", "moe_route_scored_backward",
                     "moe_combine", "moe_combine_backward", "moe_mxfp4_quantize", "moe_workspace_init",
                     "moe_get_status"}
    assert [c for c in calls if c[1:] != (1, 1001)] == []
    assert torch.cuda.current_device() == 0
