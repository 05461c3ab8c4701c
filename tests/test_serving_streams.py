"""What the serving binding allocates for a call on an explicit stream."""
import contextlib

import pytest
import torch

import dual_scale_solver_b200 as dq
from dual_scale_solver_b200 import serving


class _Recorded(torch.Tensor):
    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", []) + [stream]


@pytest.fixture
def fakes(monkeypatch):
    """The binding on CPU tensors: no library, and streams that are names.
    Yields (allocated tensors, each with the name of the stream that was
    current then; names of the streams that kernels were called on)."""
    from dual_scale_solver_b200 import build
    build.build()                                # (formats come from the library)
    current, made, called = ["current"], [], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def new(*args, **kw):
        t = torch.empty_strided(*args, **kw).as_subclass(_Recorded)
        t.owner = current[-1]
        made.append(t)
        return t

    class Library:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(serving, "_lib", lambda: Library())
    monkeypatch.setattr(serving, "_device", lambda tensors: 0)
    monkeypatch.setattr(serving, "_call", lambda device, s, fn, *a: called.append(s) or 0)
    monkeypatch.setattr(serving, "_new", new)
    monkeypatch.setattr(serving, "kv_attention_workspace", lambda *a: 512)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    return made, called


def _calls():
    f, x = dq.format_preset("mxfp4"), torch.zeros(3, 64, dtype=torch.bfloat16)
    cache = dq.kv_cache(2, 16, 2, 64, f, device="cpu")
    i = lambda *v: torch.tensor(v, dtype=torch.int32)              # noqa: E731
    meta = (i(0, 3), i(3), torch.zeros(1, 2, dtype=torch.int32))
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    return {"add_rmsnorm_quant": (3, lambda **a: dq.add_rmsnorm_quant(x, x[0], f, residual=x, **a)),
            "kv_read": (2, lambda **a: dq.kv_read(cache, *meta, f, 3, **a)),
            "kv_attention": (2, lambda **a: dq.kv_attention(q, cache, *meta, f, **a))}


@pytest.mark.parametrize("name", ["add_rmsnorm_quant", "kv_read", "kv_attention"])
def test_allocations_belong_to_the_stream_of_the_call(fakes, name):
    made, called = fakes
    count, call = _calls()[name]
    result = call(stream="side")
    assert called == ["side"] and len(made) == count
    assert [t.owner for t in made] == ["side"] * count
    for t in (result if isinstance(result, tuple) else (result,)):
        assert t.recorded == ["current"]         # the caller may drop it there
    del made[:], called[:]
    call()
    assert called == [None] and [t.owner for t in made] == ["current"] * count
    assert not any(hasattr(t, "recorded") for t in made)
